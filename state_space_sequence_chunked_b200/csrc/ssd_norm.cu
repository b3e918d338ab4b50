// The norms before and after a block, with the residual add, its scale and the gate fused in, and
// their gradients. All are single passes over the rows, bound by HBM (fractions of the measured 6.45 TB/s):
//
//   k_add_rmsnorm       r = residual + scale x,  out = w r rstd,  rstd = 1 / sqrt(mean r^2 + eps)
//   k_add_rmsnorm_bwd   dr = dres + rstd (w dout - n mean(w dout n)),  n = r rstd;
//                       dx = scale dr,  dw = sum over rows of dout n,  dscale = sum over rows of dr x
//   k_norm_gate         out = w n silu(z),  n = y rstd over groups of consecutive channels
//   k_gate_bwd          its gradient, or (kGateFirst) that of w n with n = g rstd, g = y silu(z), the
//                       order of ssd_gated_rmsnorm
//   k_col_sum           the sums over rows, from one partial row per CTA, in a fixed order
//
// Layout, the same for all: a group of gs channels belongs to tpg threads (a power of two below a
// warp, whole warps above), each holding S vectors of V channels in registers between the reduction
// and the output, so that every row is read once. A CTA covers gpc neighbouring groups of rpc rows
// at a time and walks the rows in steps of gridDim.y * rpc: its threads keep their columns, hence
// the weights and the column sums of dw and dscale stay in registers too, and no atomics are
// needed. Statistics and sums are fp32; an output that is stored in bf16 is rounded once, and the scaled
// gradient dx is rounded from dr before dr is.
//
// Measured, bf16 rows: k_add_rmsnorm 32768 x 2560, fp32 residual, 165 us a call, 94%. k_add_rmsnorm_bwd 8191 x 2560 with all
// outputs 53 us and its column sums 5.5, 66% together: two CTAs per SM hold dw and dscale in registers, and a
// third does not fit. k_norm_gate 32768 x 5120 in groups of 64, 191 us a call, 82%. k_gate_bwd 16384 x 1536 in groups of 64,
// 53 us and 5.5, 66%. The next row is loaded before the present one is reduced (gradients 71 -> 59 us
// and 62 -> 59); two rows ahead 73 and 59 (spills), loads through a ring in shared memory 10% slower (issue).
#include "ssd_norm.cuh"

namespace ssd {
namespace {

constexpr int kMaxThr = 512;
constexpr int kPer = 16;      // channels a thread may hold
constexpr int kMaxParts = 592;  // partial rows of a column sum at most: 4 CTAs on each of 148 SMs

struct Geom {
    uint32_t rows;  // below 2^31, so that a step past the end does not wrap
    int gs, ngroups, tpg, gpc, rpc;
    float inv;  // 1 / gs
};

// 1 / (1 + 2^(-v log2 e)) by the approximate instructions (2^-22 and 2^-23 of the value). The product v log2 e is
// rounded, which moves the power by up to |v| 2^-24 of itself: below -20 that is more than the rest. For outputs stored in
// bf16 it stays (5e-6 at the most, of 2^-8); for fp32 what the rounding took is multiplied back in. 0 below -87.3, where the
// quotient is no normal number. v is held within +-200, so that infinities have no remainder; a NaN v
// comes back with the factor v beside.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
    constexpr float kLog2e = 1.44269502f, kRest = 1.92596299e-8f;  // log2 e in two parts
    float e, r;
    if constexpr (sizeof(T) == 4) {
        v = fminf(fmaxf(v, -200.f), 200.f);
        const float p = -kLog2e * v, rest = fmaf(-kRest, v, fmaf(-kLog2e, v, -p));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(p));
        e *= fmaf(rest, 0.693147181f, 1.f);
    } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kLog2e * v));
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// V neighbouring channels as they lie in memory (16-byte vectors where V is 8).
template <typename T, int V>
struct Raw {
    T v[V];
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 v;
};
template <>
struct Raw<__nv_bfloat16, 2> {
    __nv_bfloat162 v;
};
template <>
struct Raw<float, 8> {
    float4 v[2];
};
template <>
struct Raw<float, 2> {
    float2 v;
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, V> *>(p);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &r, float (&f)[V]) {
    if constexpr (sizeof(T) == 2) {
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f32(e[i]);
    } else {
        const float *e = reinterpret_cast<const float *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = e[i];
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float (&f)[V]) {
    if constexpr (V == 8 && sizeof(T) == 2) {
        uint4 r;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = r;
    } else if constexpr (V == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else if constexpr (V == 2 && sizeof(T) == 2) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(f[0], f[1]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
    } else {
        store_as(p, f[0]);
    }
}

// Where this thread stands.
struct Pos {
    int tl, slot, row_slot, group;
    bool live;
    __device__ __forceinline__ explicit Pos(const Geom &q) {
        tl = threadIdx.x % q.tpg;
        slot = threadIdx.x / q.tpg;
        row_slot = slot / q.gpc;
        group = blockIdx.x * q.gpc + slot % q.gpc;
        live = group < q.ngroups && row_slot < q.rpc;
    }
};

// Sums of M values over the tpg threads of a group, returned to all of them. Every thread of the CTA
// calls it. Where a group spans warps they meet in one of two buffers in turn, so that one barrier a
// call is enough.
template <int M>
struct SumBuf {
    float v[2][M][kMaxThr / 32];
};
template <int M>
__device__ __forceinline__ void group_sum(float (&v)[M], int tpg, SumBuf<M> &buf, uint32_t &turn) {
    if (tpg <= 32) {
        for (int o = tpg >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    const int warp = threadIdx.x >> 5, wpg = tpg >> 5, first = warp / wpg * wpg;
    float(&b)[M][kMaxThr / 32] = buf.v[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) b[m][warp] = v[m];
    __syncthreads();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = lane < wpg ? b[m][first + lane] : 0.f;
#pragma unroll
    for (int o = kMaxThr / 64; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = __shfl_sync(0xffffffffu, v[m], 0);
}

template <int V, int S>
__device__ __forceinline__ void load_cols(const float *__restrict__ src, const Geom &q, const Pos &at, float (&f)[S][V],
                                          float none) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = (at.tl + s * q.tpg) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) f[s][v] = src && at.live && e < q.gs ? src[(int64_t)at.group * q.gs + e + v] : none;
    }
}

// The CTA's sum over its row slots of the threads' column sums, to row blockIdx.y of `part`.
template <int V, int S>
__device__ __forceinline__ void put_part(const float (&f)[S][V], const Geom &q, const Pos &at, float *sm, float *part) {
    const int span = q.gpc * q.gs, dim = q.gs * q.ngroups;
    __syncthreads();
    if (at.live)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (e < q.gs)
#pragma unroll
                for (int v = 0; v < V; ++v) sm[at.row_slot * span + (at.slot % q.gpc) * q.gs + e + v] = f[s][v];
        }
    __syncthreads();
    const int c0 = blockIdx.x * span;
    for (int c = threadIdx.x; c < span && c0 + c < dim; c += blockDim.x) {
        float s = 0.f;
        for (int r = 0; r < q.rpc; ++r) s += sm[r * span + c];
        part[(int64_t)blockIdx.y * dim + c0 + c] = s;
    }
}

// The rows of one step: U per thread, all of their vectors loaded before any is reduced, so that U times
// the bytes are in flight and a reduction across warps serves U rows.
#define SSD_FOR_ROWS(q, U)                                             \
    for (uint32_t base = blockIdx.y * (uint32_t)(q.rpc * U) + at.row_slot; base - at.row_slot < q.rows; \
         base += gridDim.y * (uint32_t)(q.rpc * U))

// Two rows at a time where they are read in 16-byte vectors (U = 2).
template <typename T, typename R, int V, int S, int U>
__global__ void __launch_bounds__(V == 8 && S == 1 ? 768 : kMaxThr)
    k_add_rmsnorm(Geom q, const T *x, const R *residual, const float *__restrict__ scale, const float *__restrict__ w,
                  float eps, R *res_out, T *out) {
    __shared__ SumBuf<U> buf;
    uint32_t turn = 0;
    const Pos at(q);
    float wv[S][V], sv[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
    load_cols<V, S>(scale, q, at, sv, 1.f);
    SSD_FOR_ROWS(q, U) {
        Raw<T, V> xr[U][S];
        Raw<R, V> rr[U][S];
        float sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t row = base + u * q.rpc;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int e = (at.tl + s * q.tpg) * V;
                if (at.live && row < q.rows && e < q.gs) {
                    xr[u][s] = load_raw<T, V>(x + (int64_t)row * q.gs + e);
                    if (residual) rr[u][s] = load_raw<R, V>(residual + (int64_t)row * q.gs + e);
                }
            }
        }
        float r[U][S][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t row = base + u * q.rpc;
            sum[u] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int e = (at.tl + s * q.tpg) * V;
                if (at.live && row < q.rows && e < q.gs) {
                    unpack(xr[u][s], r[u][s]);
                    if (scale) {
#pragma unroll
                        for (int v = 0; v < V; ++v) r[u][s][v] *= sv[s][v];
                    }
                    if (residual) {
                        float o[V];
                        unpack(rr[u][s], o);
#pragma unroll
                        for (int v = 0; v < V; ++v) r[u][s][v] += o[v];
                    }
                    if (res_out) store_v<R, V>(res_out + (int64_t)row * q.gs + e, r[u][s]);
#pragma unroll
                    for (int v = 0; v < V; ++v) sum[u] = fmaf(r[u][s][v], r[u][s][v], sum[u]);
                }
            }
        }
        group_sum(sum, q.tpg, buf, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t row = base + u * q.rpc;
            const float rstd = rsqrtf(fmaf(sum[u], q.inv, eps));
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int e = (at.tl + s * q.tpg) * V;
                if (at.live && row < q.rows && e < q.gs) {
#pragma unroll
                    for (int v = 0; v < V; ++v) r[u][s][v] *= rstd * wv[s][v];
                    store_v<T, V>(out + (int64_t)row * q.gs + e, r[u][s]);
                }
            }
        }
    }
}

// The other kernels keep a row as it was loaded (packed) between the two passes over it, and load the next
// row before they begin on it, so that loads are in flight all the time.
template <typename T, typename R, int V, int S>
__global__ void __launch_bounds__(V == 8 && S == 1 ? 640 : kMaxThr)
    k_add_rmsnorm_bwd(Geom q, const R *r, const float *__restrict__ w, float eps, const T *dout, const R *dres_in, const T *x,
                      const float *__restrict__ scale, R *dres, T *dx, float *dw_part, float *ds_part) {
    extern __shared__ __align__(16) float sm[];
    __shared__ SumBuf<2> buf;
    uint32_t turn = 0;
    const Pos at(q);
    float *ws = sm, *ss = sm + q.gs;
    for (int i = threadIdx.x; i < q.gs; i += blockDim.x) {
        ws[i] = w[i];
        ss[i] = scale ? scale[i] : 1.f;
    }
    float dw[S][V], ds[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[s][v] = ds[s][v] = 0.f;
    __syncthreads();
    struct Row {
        Raw<R, V> r[S], i[S];
        Raw<T, V> d[S], x[S];
    };
    const auto load = [&](Row &to, uint32_t row) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (at.live && row < q.rows && e < q.gs) {
                const int64_t off = (int64_t)row * q.gs + e;
                to.r[s] = load_raw<R, V>(r + off);
                to.d[s] = load_raw<T, V>(dout + off);
                if (dres_in) to.i[s] = load_raw<R, V>(dres_in + off);
                if (ds_part) to.x[s] = load_raw<T, V>(x + off);
            }
        }
    };
    constexpr bool kAhead = V == 8 && S == 1;
    Row next;
    if (kAhead) load(next, blockIdx.y * (uint32_t)q.rpc + at.row_slot);
    SSD_FOR_ROWS(q, 1) {
        const uint32_t row = base;
        const bool on = at.live && row < q.rows;
        Row now;
        if (kAhead) {
            now = next;
            load(next, row + gridDim.y * (uint32_t)q.rpc);
        } else {
            load(now, row);
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float rv[V], dv[V], wv[V];
                unpack(now.r[s], rv);
                unpack(now.d[s], dv);
                unpack(load_raw<float, V>(ws + e), wv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sum[0] = fmaf(rv[v], rv[v], sum[0]);
                    sum[1] = fmaf(wv[v] * dv[v], rv[v], sum[1]);
                }
            }
        }
        group_sum(sum, q.tpg, buf, turn);
        const float rstd = rsqrtf(fmaf(sum[0], q.inv, eps)), mean = sum[1] * rstd * q.inv;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float rv[V], dv[V], wv[V], o[V], xv[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = xv[v] = 0.f;
                const int64_t off = (int64_t)row * q.gs + e;
                unpack(now.r[s], rv);
                unpack(now.d[s], dv);
                unpack(load_raw<float, V>(ws + e), wv);
                if (dres_in) unpack(now.i[s], o);
                if (ds_part) unpack(now.x[s], xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float n = rv[v] * rstd;
                    dw[s][v] = fmaf(dv[v], n, dw[s][v]);
                    o[v] = fmaf(rstd, fmaf(-n, mean, wv[v] * dv[v]), o[v]);
                    ds[s][v] = fmaf(o[v], xv[v], ds[s][v]);
                }
                if (dres) store_v<R, V>(dres + off, o);
                if (dx) {
                    unpack(load_raw<float, V>(ss + e), wv);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] *= wv[v];
                    store_v<T, V>(dx + off, o);
                }
            }
        }
    }
    if (dw_part) put_part<V, S>(dw, q, at, sm, dw_part);
    if (ds_part) put_part<V, S>(ds, q, at, sm, ds_part);
}

template <typename T, int V, int S>
__global__ void __launch_bounds__(V == 8 && S == 1 ? 1024 : kMaxThr)
    k_norm_gate(Geom q, const T *y, const T *z, int64_t z_stride, const float *__restrict__ w, float eps, T *out) {
    __shared__ SumBuf<1> buf;
    uint32_t turn = 0;
    const Pos at(q);
    const int dim = q.gs * q.ngroups, col = at.group * q.gs;
    float wv[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
    struct Row {
        Raw<T, V> y[S], z[S];
    };
    const auto load = [&](Row &to, uint32_t row) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (at.live && row < q.rows && e < q.gs) {
                to.y[s] = load_raw<T, V>(y + (int64_t)row * dim + (col + e));
                to.z[s] = load_raw<T, V>(z + (int64_t)row * z_stride + (col + e));
            }
        }
    };
    constexpr bool kAhead = V == 8 && S == 1;
    Row next;
    if (kAhead) load(next, blockIdx.y * (uint32_t)q.rpc + at.row_slot);
    SSD_FOR_ROWS(q, 1) {
        const uint32_t row = base;
        const bool on = at.live && row < q.rows;
        Row now;
        if (kAhead) {
            now = next;
            load(next, row + gridDim.y * (uint32_t)q.rpc);
        } else {
            load(now, row);
        }
        float sum[1] = {0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float f[V];
                unpack(now.y[s], f);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[0] = fmaf(f[v], f[v], sum[0]);
            }
        }
        group_sum(sum, q.tpg, buf, turn);
        const float rstd = rsqrtf(fmaf(sum[0], q.inv, eps));
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float f[V], zv[V];
                unpack(now.y[s], f);
                unpack(now.z[s], zv);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] *= (rstd * wv[s][v]) * (zv[v] * sigmoid<T>(zv[v]));
                store_v<T, V>(out + (int64_t)row * dim + (col + e), f);
            }
        }
    }
}

template <typename T, int V, int S, bool kGateFirst>
__global__ void __launch_bounds__(V == 8 && S == 1 ? 640 : kMaxThr)
    k_gate_bwd(Geom q, const T *y, const T *z, int64_t z_stride, const float *__restrict__ w, float eps, const T *dout, T *dy,
               T *dz, int64_t dz_stride, float *dw_part) {
    extern __shared__ __align__(16) float sm[];
    __shared__ SumBuf<2> buf;
    uint32_t turn = 0;
    const Pos at(q);
    const int dim = q.gs * q.ngroups, col = at.group * q.gs;
    float wv[S][V], dw[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[s][v] = 0.f;
    struct Row {
        Raw<T, V> y[S], z[S], d[S];
    };
    const auto load = [&](Row &to, uint32_t row) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (at.live && row < q.rows && e < q.gs) {
                to.y[s] = load_raw<T, V>(y + (int64_t)row * dim + (col + e));
                to.z[s] = load_raw<T, V>(z + (int64_t)row * z_stride + (col + e));
                to.d[s] = load_raw<T, V>(dout + (int64_t)row * dim + (col + e));
            }
        }
    };
    constexpr bool kAhead = V == 8 && S == 1;
    Row next;
    if (kAhead) load(next, blockIdx.y * (uint32_t)q.rpc + at.row_slot);
    SSD_FOR_ROWS(q, 1) {
        const uint32_t row = base;
        const bool on = at.live && row < q.rows;
        Row now;
        if (kAhead) {
            now = next;
            load(next, row + gridDim.y * (uint32_t)q.rpc);
        } else {
            load(now, row);
        }
        float sg[S][V], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float yv[V], zv[V], dv[V];
                unpack(now.y[s], yv);
                unpack(now.z[s], zv);
                unpack(now.d[s], dv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sg[s][v] = sigmoid<T>(zv[v]);
                    const float gate = zv[v] * sg[s][v];
                    const float a = kGateFirst ? yv[v] * gate : yv[v];             // what is normalised
                    const float b = wv[s][v] * dv[v] * (kGateFirst ? 1.f : gate);  // its cotangent
                    sum[0] = fmaf(a, a, sum[0]);
                    sum[1] = fmaf(a, b, sum[1]);
                }
            }
        }
        group_sum(sum, q.tpg, buf, turn);
        const float rstd = rsqrtf(fmaf(sum[0], q.inv, eps)), mean = sum[1] * rstd * q.inv;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float yv[V], zv[V], dv[V], oy[V], oz[V];
                unpack(now.y[s], yv);
                unpack(now.z[s], zv);
                unpack(now.d[s], dv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sig = sg[s][v], gate = zv[v] * sig;
                    const float slope = sig * fmaf(zv[v], 1.f - sig, 1.f);
                    if constexpr (kGateFirst) {
                        const float n = yv[v] * gate * rstd, d = rstd * (wv[s][v] * dv[v] - n * mean);
                        dw[s][v] = fmaf(dv[v], n, dw[s][v]);
                        oy[v] = d * gate;
                        oz[v] = d * yv[v] * slope;
                    } else {
                        const float n = yv[v] * rstd, dn = dv[v] * n;
                        dw[s][v] = fmaf(dn, gate, dw[s][v]);
                        oy[v] = rstd * (wv[s][v] * dv[v] * gate - n * mean);
                        oz[v] = wv[s][v] * dn * slope;
                    }
                }
                store_v<T, V>(dy + (int64_t)row * dim + (col + e), oy);
                store_v<T, V>(dz + (int64_t)row * dz_stride + (col + e), oz);
            }
        }
    }
    if (dw_part) put_part<V, S>(dw, q, at, sm, dw_part);
}

// out[c] = sum over the partial rows, in order per thread row; grid.y picks the first or second sum.
// grid (ceil(dim / 32), 1 or 2), (32, 32) threads.
__global__ void k_col_sum(const float *__restrict__ part, int parts, int dim, float *__restrict__ out0,
                          float *__restrict__ out1) {
    __shared__ float sm[32][33];
    float *out = blockIdx.y ? out1 : out0;
    part += (int64_t)blockIdx.y * parts * dim;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < dim)
#pragma unroll 4
        for (int r = threadIdx.y; r < parts; r += 32) s += part[(int64_t)r * dim + c];
    sm[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        float t = 0.f;
        for (int r = 0; r < 32; ++r) t += sm[r][threadIdx.x];
        out[c] = t;
    }
}

// Vector width: 8 channels where groups, strides and pointers allow 16-byte bf16 (32-byte fp32)
// vectors, 2 where they allow pairs, else 1.
int vec_of(int64_t gs, int64_t stride_a, int64_t stride_b, size_t es, std::initializer_list<const void *> ptrs) {
    const auto fits = [&](int64_t n, size_t bytes) {
        bool ok = gs % n == 0 && stride_a % n == 0 && stride_b % n == 0;
        for (const void *p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % bytes == 0;
        return ok;
    };
    return fits(8, 16) ? 8 : fits(2, 2 * es) ? 2 : 1;
}

struct Launch {
    Geom q;
    dim3 grid;
    int threads;
    size_t smem;
    cudaError_t error;
};

// One wave of `kernel`: as many CTAs as fit on the SMs at once, each walking its share of the rows.
template <typename K>
Launch geom(K kernel, int64_t rows, int gs, int ngroups, int V, int S, int U, size_t smem) {
    Launch l{};
    const int nvec = (gs + V - 1) / V, need = (nvec + S - 1) / S;
    int tpg = 1;
    if (need <= 32)
        while (tpg < need) tpg <<= 1;
    else
        tpg = (need + 31) / 32 * 32;
    const int slots = tpg >= 256 ? 1 : 256 / tpg;
    const int gpc = ngroups < slots ? ngroups : slots;
    int rpc = slots / gpc;
    if (rpc > rows) rpc = (int)rows;
    const int thr = (tpg * gpc * rpc + 31) / 32 * 32;
    const int gx = (ngroups + gpc - 1) / gpc;
    // the backward kernels' column sums pass through shared memory, rpc rows of gpc groups
    l.smem = smem;
    if (smem && l.smem < (size_t)rpc * gpc * gs * sizeof(float)) l.smem = (size_t)rpc * gpc * gs * sizeof(float);
    l.error = l.smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)l.smem) : cudaSuccess;
    int fit = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, thr, l.smem) != cudaSuccess || fit < 1) fit = 1;
    int64_t gy = (rows + rpc * U - 1) / (rpc * U);
    const int64_t wave = (int64_t)sm_count() * fit, most = wave / gx > 1 ? wave / gx : 1;
    if (gy > most) gy = most;
    if (gy > kMaxParts) gy = kMaxParts;
    l.q = Geom{(uint32_t)rows, gs, ngroups, tpg, gpc, rpc, (float)(1.0 / gs)};
    l.grid = dim3((unsigned)gx, (unsigned)gy);
    l.threads = thr;
    return l;
}

// Calls f with (V, S) as constants: as few vectors per thread as the group needs.
template <int V_, int S_>
struct VS {
    static constexpr int V = V_, S = S_, U = V_ == 8 && S_ == 1 ? 2 : 1;
};
template <typename F>
cudaError_t with_vs(int vec, int gs, F f) {
    if (vec == 8) return gs <= 8 * kMaxThr ? f(VS<8, 1>()) : f(VS<8, 2>());
    if (vec == 2) return gs <= 4 * kMaxThr ? f(VS<2, 2>()) : f(VS<2, 8>());
    return gs <= 4 * kMaxThr ? f(VS<1, 4>()) : f(VS<1, 16>());
}

// Sums of one or two partial arrays that follow one another; out1 may be NULL.
cudaError_t col_sum(const float *part, int parts, int dim, float *out0, float *out1, cudaStream_t s) {
    k_col_sum<<<dim3((dim + 31) / 32, out1 ? 2 : 1), dim3(32, 32), 0, s>>>(part, parts, dim, out0, out1);
    return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t add_fwd(const AddNormArgs &a, cudaStream_t st) {
    const int vec = vec_of(a.dim, a.dim, a.dim, 4, {a.x, a.residual, a.res_out, a.out});
    return with_vs(vec, (int)a.dim, [&](auto vs) {
        const auto kernel = k_add_rmsnorm<T, R, vs.V, vs.S, vs.U>;
        const Launch l = geom(kernel, a.rows, (int)a.dim, 1, vs.V, vs.S, vs.U, 0);
        if (l.error) return l.error;
        kernel<<<l.grid, l.threads, l.smem, st>>>(
            l.q, static_cast<const T *>(a.x), static_cast<const R *>(a.residual), a.scale, a.weight, a.eps,
            static_cast<R *>(a.res_out), static_cast<T *>(a.out));
        return cudaGetLastError();
    });
}

template <typename T, typename R>
cudaError_t add_bwd(const AddNormArgs &a, const AddNormGrads &g, float *ws, cudaStream_t st) {
    const int vec = vec_of(a.dim, a.dim, a.dim, 4, {a.residual, g.dout, g.dres_in, a.x, g.dres, g.dx});
    return with_vs(vec, (int)a.dim, [&](auto vs) {
        const auto kernel = k_add_rmsnorm_bwd<T, R, vs.V, vs.S>;
        const Launch l = geom(kernel, a.rows, (int)a.dim, 1, vs.V, vs.S, 1, 8 * (size_t)a.dim);
        if (l.error) return l.error;
        float *dw = g.dw ? ws : nullptr, *ds = g.dscale ? (dw ? ws + (int64_t)l.grid.y * a.dim : ws) : nullptr;
        kernel<<<l.grid, l.threads, l.smem, st>>>(
            l.q, static_cast<const R *>(a.residual), a.weight, a.eps, static_cast<const T *>(g.dout),
            static_cast<const R *>(g.dres_in), static_cast<const T *>(a.x), a.scale, static_cast<R *>(g.dres),
            static_cast<T *>(g.dx), dw, ds);
        cudaError_t e = cudaGetLastError();
        if (!e && (dw || ds))
            e = col_sum(ws, (int)l.grid.y, (int)a.dim, dw ? g.dw : g.dscale, dw ? g.dscale : nullptr, st);
        return e;
    });
}

template <typename T>
cudaError_t gate_fwd(const GateNormArgs &a, cudaStream_t st) {
    const int gs = (int)(a.dim / a.ngroups);
    const int vec = vec_of(gs, a.z_stride, gs, sizeof(T), {a.y, a.z, a.out});
    return with_vs(vec, gs, [&](auto vs) {
        const auto kernel = k_norm_gate<T, vs.V, vs.S>;
        const Launch l = geom(kernel, a.rows, gs, (int)a.ngroups, vs.V, vs.S, 1, 0);
        if (l.error) return l.error;
        kernel<<<l.grid, l.threads, l.smem, st>>>(l.q, static_cast<const T *>(a.y), static_cast<const T *>(a.z), a.z_stride,
                                                  a.weight, a.eps, static_cast<T *>(a.out));
        return cudaGetLastError();
    });
}

template <typename T, bool kGateFirst>
cudaError_t gate_bwd(const GateNormArgs &a, const GateNormGrads &g, float *ws, cudaStream_t st) {
    const int gs = (int)(a.dim / a.ngroups);
    const int vec = vec_of(gs, a.z_stride, g.dz_stride, sizeof(T), {a.y, a.z, g.dout, g.dy, g.dz});
    return with_vs(vec, gs, [&](auto vs) {
        const auto kernel = k_gate_bwd<T, vs.V, vs.S, kGateFirst>;
        const Launch l = geom(kernel, a.rows, gs, (int)a.ngroups, vs.V, vs.S, 1, 4);
        if (l.error) return l.error;
        float *dw = g.dw ? ws : nullptr;
        kernel<<<l.grid, l.threads, l.smem, st>>>(
            l.q, static_cast<const T *>(a.y), static_cast<const T *>(a.z), a.z_stride, a.weight, a.eps,
            static_cast<const T *>(g.dout), static_cast<T *>(g.dy), static_cast<T *>(g.dz), g.dz_stride, dw);
        cudaError_t e = cudaGetLastError();
        if (!e && dw) e = col_sum(dw, (int)l.grid.y, (int)a.dim, g.dw, nullptr, st);
        return e;
    });
}

}  // namespace

int norm_max_group() { return kMaxThr * kPer; }

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    return (size_t)(rows < kMaxParts ? rows : kMaxParts) * (size_t)dim * 2 * sizeof(float);
}

cudaError_t add_rmsnorm_launch(const AddNormArgs &a, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (a.dtype == SSD_F32) return add_fwd<float, float>(a, s);
    return a.res_dtype == SSD_F32 ? add_fwd<bf, float>(a, s) : add_fwd<bf, bf>(a, s);
}

cudaError_t add_rmsnorm_bwd_launch(const AddNormArgs &a, const AddNormGrads &g, float *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (a.dtype == SSD_F32) return add_bwd<float, float>(a, g, ws, s);
    return a.res_dtype == SSD_F32 ? add_bwd<bf, float>(a, g, ws, s) : add_bwd<bf, bf>(a, g, ws, s);
}

cudaError_t norm_gate_launch(const GateNormArgs &a, cudaStream_t s) {
    return a.dtype == SSD_F32 ? gate_fwd<float>(a, s) : gate_fwd<__nv_bfloat16>(a, s);
}

cudaError_t gate_norm_bwd_launch(const GateNormArgs &a, const GateNormGrads &g, bool gate_first, float *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (a.dtype == SSD_F32) return gate_first ? gate_bwd<float, true>(a, g, ws, s) : gate_bwd<float, false>(a, g, ws, s);
    return gate_first ? gate_bwd<bf, true>(a, g, ws, s) : gate_bwd<bf, false>(a, g, ws, s);
}

}  // namespace ssd
