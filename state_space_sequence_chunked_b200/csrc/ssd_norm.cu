// The norms before and after a block, with the residual add, its scale and the gate fused in, and
// their gradients. All are single passes over the rows, bound by HBM:
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
// needed. Statistics and sums are fp32.
#include "ssd_norm.cuh"

namespace ssd {
namespace {

constexpr int kMaxThr = 512;
constexpr int kPer = 16;      // channels a thread may hold
constexpr int kMaxParts = 592;  // partial rows of a column sum: 4 CTAs per SM

struct Geom {
    int64_t rows;
    int gs, ngroups, tpg, gpc, rpc;
};

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

template <typename T, int V>
__device__ __forceinline__ void load_v(const T *p, float (&f)[V]) {
    if constexpr (V == 8 && sizeof(T) == 2) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    } else if constexpr (V == 8) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else if constexpr (V == 2 && sizeof(T) == 2) {
        const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
        f[0] = v.x, f[1] = v.y;
    } else if constexpr (V == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        f[0] = v.x, f[1] = v.y;
    } else {
        f[0] = to_f32(p[0]);
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
// calls it (a warp of shared memory per value where a group spans warps).
template <int M>
__device__ __forceinline__ void group_sum(float (&v)[M], int tpg, float (*buf)[kMaxThr / 32]) {
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
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) buf[m][warp] = v[m];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
        float s = 0.f;
        for (int w = 0; w < wpg; ++w) s += buf[m][first + w];
        v[m] = s;
    }
    __syncthreads();
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

template <typename T, typename R, int V, int S>
__global__ void __launch_bounds__(kMaxThr)
    k_add_rmsnorm(Geom q, const T *x, const R *residual, const float *__restrict__ scale, const float *__restrict__ w,
                  float eps, R *res_out, T *out) {
    __shared__ float buf[1][kMaxThr / 32];
    const Pos at(q);
    float wv[S][V], sv[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
    load_cols<V, S>(scale, q, at, sv, 1.f);
    for (int64_t base = (int64_t)blockIdx.y * q.rpc; base < q.rows; base += (int64_t)gridDim.y * q.rpc) {
        const int64_t row = base + at.row_slot;
        const bool on = at.live && row < q.rows;
        float r[S][V], sum[1] = {0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                load_v<T, V>(x + row * q.gs + e, r[s]);
                if (residual) {
                    float o[V];
                    load_v<R, V>(residual + row * q.gs + e, o);
#pragma unroll
                    for (int v = 0; v < V; ++v) r[s][v] = scale ? fmaf(sv[s][v], r[s][v], o[v]) : r[s][v] + o[v];
                } else if (scale) {
#pragma unroll
                    for (int v = 0; v < V; ++v) r[s][v] *= sv[s][v];
                }
                if (res_out) store_v<R, V>(res_out + row * q.gs + e, r[s]);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[0] = fmaf(r[s][v], r[s][v], sum[0]);
            }
        }
        group_sum(sum, q.tpg, buf);
        const float rstd = rsqrtf(sum[0] / (float)q.gs + eps);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
#pragma unroll
                for (int v = 0; v < V; ++v) r[s][v] *= rstd * wv[s][v];
                store_v<T, V>(out + row * q.gs + e, r[s]);
            }
        }
    }
}

template <typename T, typename R, int V, int S>
__global__ void __launch_bounds__(kMaxThr)
    k_add_rmsnorm_bwd(Geom q, const R *__restrict__ r, const float *__restrict__ w, float eps, const T *dout,
                      const R *dres_in, const T *__restrict__ x, const float *__restrict__ scale, R *dres, T *dx,
                      float *dw_part, float *ds_part) {
    extern __shared__ float sm[];
    __shared__ float buf[2][kMaxThr / 32];
    const Pos at(q);
    float wv[S][V], sv[S][V], dw[S][V], ds[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
    load_cols<V, S>(scale, q, at, sv, 1.f);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[s][v] = ds[s][v] = 0.f;
    for (int64_t base = (int64_t)blockIdx.y * q.rpc; base < q.rows; base += (int64_t)gridDim.y * q.rpc) {
        const int64_t row = base + at.row_slot;
        const bool on = at.live && row < q.rows;
        float rv[S][V], dv[S][V], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                load_v<R, V>(r + row * q.gs + e, rv[s]);
                load_v<T, V>(dout + row * q.gs + e, dv[s]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sum[0] = fmaf(rv[s][v], rv[s][v], sum[0]);
                    sum[1] = fmaf(wv[s][v] * dv[s][v], rv[s][v], sum[1]);
                }
            }
        }
        group_sum(sum, q.tpg, buf);
        const float rstd = rsqrtf(sum[0] / (float)q.gs + eps), mean = sum[1] * rstd / (float)q.gs;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float o[V], xv[V];
                const int64_t off = row * q.gs + e;
                if (dres_in) load_v<R, V>(dres_in + off, o);
                if (ds_part) load_v<T, V>(x + off, xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float n = rv[s][v] * rstd;
                    dw[s][v] = fmaf(dv[s][v], n, dw[s][v]);
                    const float d = rstd * (wv[s][v] * dv[s][v] - n * mean);
                    o[v] = dres_in ? o[v] + d : d;
                    if (ds_part) ds[s][v] = fmaf(o[v], xv[v], ds[s][v]);
                }
                if (dres) store_v<R, V>(dres + off, o);
                if (dx) {
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] *= sv[s][v];
                    store_v<T, V>(dx + off, o);
                }
            }
        }
    }
    if (dw_part) put_part<V, S>(dw, q, at, sm, dw_part);
    if (ds_part) put_part<V, S>(ds, q, at, sm, ds_part);
}

template <typename T, int V, int S>
__global__ void __launch_bounds__(kMaxThr)
    k_norm_gate(Geom q, const T *y, const T *__restrict__ z, int64_t z_stride, const float *__restrict__ w, float eps,
                T *out) {
    __shared__ float buf[1][kMaxThr / 32];
    const Pos at(q);
    const int dim = q.gs * q.ngroups;
    float wv[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
    for (int64_t base = (int64_t)blockIdx.y * q.rpc; base < q.rows; base += (int64_t)gridDim.y * q.rpc) {
        const int64_t row = base + at.row_slot;
        const bool on = at.live && row < q.rows;
        const int col = at.group * q.gs;
        float f[S][V], zv[S][V], sum[1] = {0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                load_v<T, V>(y + row * dim + col + e, f[s]);
                load_v<T, V>(z + row * z_stride + col + e, zv[s]);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[0] = fmaf(f[s][v], f[s][v], sum[0]);
            }
        }
        group_sum(sum, q.tpg, buf);
        const float rstd = rsqrtf(sum[0] / (float)q.gs + eps);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
#pragma unroll
                for (int v = 0; v < V; ++v) f[s][v] *= rstd * wv[s][v] * zv[s][v] * sigmoid(zv[s][v]);
                store_v<T, V>(out + row * dim + col + e, f[s]);
            }
        }
    }
}

template <typename T, int V, int S, bool kGateFirst>
__global__ void __launch_bounds__(kMaxThr)
    k_gate_bwd(Geom q, const T *y, const T *z, int64_t z_stride, const float *__restrict__ w, float eps, const T *dout, T *dy,
               T *dz, int64_t dz_stride, float *dw_part) {
    extern __shared__ float sm[];
    __shared__ float buf[2][kMaxThr / 32];
    const Pos at(q);
    const int dim = q.gs * q.ngroups;
    float wv[S][V], dw[S][V];
    load_cols<V, S>(w, q, at, wv, 0.f);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[s][v] = 0.f;
    for (int64_t base = (int64_t)blockIdx.y * q.rpc; base < q.rows; base += (int64_t)gridDim.y * q.rpc) {
        const int64_t row = base + at.row_slot;
        const bool on = at.live && row < q.rows;
        const int col = at.group * q.gs;
        float yv[S][V], zv[S][V], dv[S][V], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                load_v<T, V>(y + row * dim + col + e, yv[s]);
                load_v<T, V>(z + row * z_stride + col + e, zv[s]);
                load_v<T, V>(dout + row * dim + col + e, dv[s]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float gate = zv[s][v] * sigmoid(zv[s][v]);
                    const float a = kGateFirst ? yv[s][v] * gate : yv[s][v];  // what is normalised
                    const float b = wv[s][v] * dv[s][v] * (kGateFirst ? 1.f : gate);  // its cotangent
                    sum[0] = fmaf(a, a, sum[0]);
                    sum[1] = fmaf(a, b, sum[1]);
                }
            }
        }
        group_sum(sum, q.tpg, buf);
        const float rstd = rsqrtf(sum[0] / (float)q.gs + eps), mean = sum[1] * rstd / (float)q.gs;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (at.tl + s * q.tpg) * V;
            if (on && e < q.gs) {
                float oy[V], oz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sig = sigmoid(zv[s][v]), gate = zv[s][v] * sig;
                    const float slope = sig * fmaf(zv[s][v], 1.f - sig, 1.f);
                    if constexpr (kGateFirst) {
                        const float n = yv[s][v] * gate * rstd, d = rstd * (wv[s][v] * dv[s][v] - n * mean);
                        dw[s][v] = fmaf(dv[s][v], n, dw[s][v]);
                        oy[v] = d * gate;
                        oz[v] = d * yv[s][v] * slope;
                    } else {
                        const float n = yv[s][v] * rstd, dn = dv[s][v] * n;
                        dw[s][v] = fmaf(dn, gate, dw[s][v]);
                        oy[v] = rstd * (wv[s][v] * dv[s][v] * gate - n * mean);
                        oz[v] = wv[s][v] * dn * slope;
                    }
                }
                store_v<T, V>(dy + row * dim + col + e, oy);
                store_v<T, V>(dz + row * dz_stride + col + e, oz);
            }
        }
    }
    if (dw_part) put_part<V, S>(dw, q, at, sm, dw_part);
}

// out[c] = sum over the partial rows, in order per thread row. grid (ceil(dim / 32)), (32, 32) threads.
__global__ void k_col_sum(const float *__restrict__ part, int parts, int dim, float *__restrict__ out) {
    __shared__ float sm[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < dim)
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
    size_t smem;  // of put_part
};

Launch geom(int64_t rows, int gs, int ngroups, int V, int S) {
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
    const int64_t want = 148 * (2048 / thr > 1 ? 2048 / thr : 1), most = (want + gx - 1) / gx;
    int64_t gy = (rows + rpc - 1) / rpc;
    if (gy > most) gy = most;
    if (gy > kMaxParts) gy = kMaxParts;
    l.q = Geom{rows, gs, ngroups, tpg, gpc, rpc};
    l.grid = dim3((unsigned)gx, (unsigned)gy);
    l.threads = thr;
    l.smem = (size_t)rpc * gpc * gs * sizeof(float);
    return l;
}

// Calls f with (V, S) as constants: V = 8 holds 1 or 2 vectors, V = 2 eight, V = 1 sixteen.
template <int V_, int S_>
struct VS {
    static constexpr int V = V_, S = S_;
};
template <typename F>
cudaError_t with_vs(int vec, int gs, F f) {
    if (vec == 8) return gs <= 8 * kMaxThr ? f(VS<8, 1>()) : f(VS<8, 2>());
    return vec == 2 ? f(VS<2, 8>()) : f(VS<1, 16>());
}

cudaError_t col_sum(const float *part, int parts, int dim, float *out, cudaStream_t s) {
    k_col_sum<<<(dim + 31) / 32, dim3(32, 32), 0, s>>>(part, parts, dim, out);
    return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t add_fwd(const AddNormArgs &a, cudaStream_t st) {
    const int vec = vec_of(a.dim, a.dim, a.dim, 4, {a.x, a.residual, a.res_out, a.out});
    return with_vs(vec, (int)a.dim, [&](auto vs) {
        const Launch l = geom(a.rows, (int)a.dim, 1, vs.V, vs.S);
        k_add_rmsnorm<T, R, vs.V, vs.S><<<l.grid, l.threads, 0, st>>>(
            l.q, static_cast<const T *>(a.x), static_cast<const R *>(a.residual), a.scale, a.weight, a.eps,
            static_cast<R *>(a.res_out), static_cast<T *>(a.out));
        return cudaGetLastError();
    });
}

template <typename T, typename R>
cudaError_t add_bwd(const AddNormArgs &a, const AddNormGrads &g, float *ws, cudaStream_t st) {
    const int vec = vec_of(a.dim, a.dim, a.dim, 4, {a.residual, g.dout, g.dres_in, a.x, g.dres, g.dx});
    return with_vs(vec, (int)a.dim, [&](auto vs) {
        const Launch l = geom(a.rows, (int)a.dim, 1, vs.V, vs.S);
        float *dw = g.dw ? ws : nullptr, *ds = g.dscale ? ws + (int64_t)l.grid.y * a.dim : nullptr;
        k_add_rmsnorm_bwd<T, R, vs.V, vs.S><<<l.grid, l.threads, l.smem, st>>>(
            l.q, static_cast<const R *>(a.residual), a.weight, a.eps, static_cast<const T *>(g.dout),
            static_cast<const R *>(g.dres_in), static_cast<const T *>(a.x), a.scale, static_cast<R *>(g.dres),
            static_cast<T *>(g.dx), dw, ds);
        cudaError_t e = cudaGetLastError();
        if (!e && dw) e = col_sum(dw, (int)l.grid.y, (int)a.dim, g.dw, st);
        if (!e && ds) e = col_sum(ds, (int)l.grid.y, (int)a.dim, g.dscale, st);
        return e;
    });
}

template <typename T>
cudaError_t gate_fwd(const GateNormArgs &a, cudaStream_t st) {
    const int gs = (int)(a.dim / a.ngroups);
    const int vec = vec_of(gs, a.z_stride, gs, sizeof(T), {a.y, a.z, a.out});
    return with_vs(vec, gs, [&](auto vs) {
        const Launch l = geom(a.rows, gs, (int)a.ngroups, vs.V, vs.S);
        k_norm_gate<T, vs.V, vs.S><<<l.grid, l.threads, 0, st>>>(l.q, static_cast<const T *>(a.y),
                                                                 static_cast<const T *>(a.z), a.z_stride, a.weight, a.eps,
                                                                 static_cast<T *>(a.out));
        return cudaGetLastError();
    });
}

template <typename T, bool kGateFirst>
cudaError_t gate_bwd(const GateNormArgs &a, const GateNormGrads &g, float *ws, cudaStream_t st) {
    const int gs = (int)(a.dim / a.ngroups);
    const int vec = vec_of(gs, a.z_stride, g.dz_stride, sizeof(T), {a.y, a.z, g.dout, g.dy, g.dz});
    return with_vs(vec, gs, [&](auto vs) {
        const Launch l = geom(a.rows, gs, (int)a.ngroups, vs.V, vs.S);
        float *dw = g.dw ? ws : nullptr;
        k_gate_bwd<T, vs.V, vs.S, kGateFirst><<<l.grid, l.threads, l.smem, st>>>(
            l.q, static_cast<const T *>(a.y), static_cast<const T *>(a.z), a.z_stride, a.weight, a.eps,
            static_cast<const T *>(g.dout), static_cast<T *>(g.dy), static_cast<T *>(g.dz), g.dz_stride, dw);
        cudaError_t e = cudaGetLastError();
        if (!e && dw) e = col_sum(dw, (int)l.grid.y, (int)a.dim, g.dw, st);
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
