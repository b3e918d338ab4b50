// The gated delta rule: its general path (any headdim, dstate <= 256, fp32 and bf16) and the
// one-token step. Per (b, h), with group k = B_t, q = C_t and a_t = exp(g_t):
//     h' = a_t h_{t-1},  err_t = x_t - h' k_t,  u_t = beta_t err_t,  h_t = h' + u_t k_t^T,  y_t = h_t q_t.
// The rows p of the state are independent given k and q: a row is h_t[p, :] = a_t h[p, :] + u_t[p] k_t,
// so a warp keeps whole rows in registers and nothing crosses warps.
//
//   k_delta_seq       token by token, a lane holding dstate / 32 columns of 2 rows. Both dot products of
//                     a token are of the state before it: y_t = a (h q) + u (k.q), so that the chain
//                     per token is one reduction and one update. For the backward pass it also
//                     leaves err and the state entering each segment of kSeg tokens.
//   k_delta_seq_bwd   the same walk in reverse: with D the cotangent of h_t,
//                     D += dy_t q_t^T, z_t = D k_t, dx_t = beta_t z_t, D <- a_t (D - dx_t k_t^T).
//                     It needs no state; it leaves z and the cotangent leaving each segment.
//   k_delta_grads     per segment, everything that sums over the rows of the state (dB, dC, dg,
//                     dbeta), from the segment's entering state, leaving cotangent, err and z.
//   k_delta_step      one token, HBM-bound: the state is read and written once.
//
// This is the exact path (fp32 throughout), bound by the latency of the token chain and not by a
// unit; bf16 inputs of the usual sizes take the chunked tensor-core path in ssd_delta_mma.cu.
#include "ssd_delta.cuh"

namespace ssd {
namespace {

constexpr int kThr = 256, kWarps = kThr / 32;
constexpr int kRows = 2;  // state rows per warp of the sequential kernels
constexpr int kTb = 16;   // tokens staged at a time

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Stages kTb tokens from t0 (zeros past L): keys, queries as fp32 rows of NJ * 32 columns.
template <typename T, int NJ>
__device__ __forceinline__ void stage_rows(const T *__restrict__ src, int64_t L, int64_t t0, int G, int N, int b, int grp,
                                           float *dst) {
    for (int i = threadIdx.x; i < kTb * NJ * 32; i += kThr) {
        const int t = i / (NJ * 32), n = i % (NJ * 32);
        const int64_t tt = t0 + t;
        dst[i] = n < N && tt < L ? to_f32(src[(((int64_t)b * L + tt) * G + grp) * N + n]) : 0.f;
    }
}

// grid (ceil(P / 16), H, B).
template <typename T, int NJ>
__global__ void __launch_bounds__(kThr)
    k_delta_seq(const T *__restrict__ x, const T *__restrict__ g, const T *__restrict__ beta, const T *__restrict__ Bm,
                const T *__restrict__ Cm, const float *__restrict__ h0, int64_t L, int H, int P, int G, int N,
                T *__restrict__ y, float *__restrict__ h_final, float *__restrict__ seg_states,
                float *__restrict__ err_out) {
    __shared__ float ks[kTb * NJ * 32], qs[kTb * NJ * 32], xs[kTb * kWarps * kRows], as[kTb], bs[kTb], kqs[kTb];
    const int h = blockIdx.y, b = blockIdx.z, grp = h / (H / G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pc = blockIdx.x * kWarps * kRows, p0 = pc + warp * kRows;
    const int64_t row0 = ((int64_t)b * H + h) * P, ns = (L + kSeg - 1) / kSeg;
    float s[kRows][NJ];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = lane + 32 * j;
            s[r][j] = h0 && p0 + r < P && n < N ? h0[(row0 + p0 + r) * N + n] : 0.f;
        }
    for (int64_t t0 = 0; t0 < L; t0 += kTb) {
        __syncthreads();
        stage_rows<T, NJ>(Bm, L, t0, G, N, b, grp, ks);
        if (Cm) stage_rows<T, NJ>(Cm, L, t0, G, N, b, grp, qs);
        for (int i = tid; i < kTb * kWarps * kRows; i += kThr) {
            const int t = i / (kWarps * kRows), p = pc + i % (kWarps * kRows);
            xs[i] = t0 + t < L && p < P ? to_f32(x[(((int64_t)b * L + t0 + t) * H + h) * P + p]) : 0.f;
        }
        if (tid < kTb && t0 + tid < L) {
            as[tid] = expf(to_f32(g[((int64_t)b * L + t0 + tid) * H + h]));
            bs[tid] = to_f32(beta[((int64_t)b * L + t0 + tid) * H + h]);
        }
        __syncthreads();
        if (Cm) {
            for (int t = warp; t < kTb; t += kWarps) {
                float d = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    d = fmaf(ks[t * NJ * 32 + lane + 32 * j], qs[t * NJ * 32 + lane + 32 * j], d);
                d = warp_sum(d);
                if (lane == 0) kqs[t] = d;
            }
            __syncthreads();
        }
        const int nt = L - t0 < kTb ? (int)(L - t0) : kTb;
        for (int t = 0; t < nt; ++t) {
            if (seg_states && (t0 + t) % kSeg == 0) {
                const int64_t c = (t0 + t) / kSeg;
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int n = lane + 32 * j;
                        if (p0 + r < P && n < N)
                            seg_states[((((int64_t)b * H + h) * ns + c) * P + p0 + r) * N + n] = s[r][j];
                    }
            }
            const float a = as[t], bt = bs[t];
            float pk[kRows], pq[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                pk[r] = pq[r] = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    pk[r] = fmaf(s[r][j], ks[t * NJ * 32 + lane + 32 * j], pk[r]);
                    if (Cm) pq[r] = fmaf(s[r][j], qs[t * NJ * 32 + lane + 32 * j], pq[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float err = xs[t * kWarps * kRows + warp * kRows + r] - a * warp_sum(pk[r]);
                const float u = bt * err;
#pragma unroll
                for (int j = 0; j < NJ; ++j) s[r][j] = fmaf(a, s[r][j], u * ks[t * NJ * 32 + lane + 32 * j]);
                const int64_t at = (((int64_t)b * L + t0 + t) * H + h) * P + p0 + r;
                if (Cm) {
                    const float yv = a * warp_sum(pq[r]) + u * kqs[t];
                    if (lane == 0 && p0 + r < P) store_as(y + at, yv);
                }
                if (err_out && lane == 0 && p0 + r < P) err_out[at] = err;
            }
        }
    }
    if (h_final) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = lane + 32 * j;
                if (p0 + r < P && n < N) h_final[(row0 + p0 + r) * N + n] = s[r][j];
            }
    }
}

// grid (ceil(P / 16), H, B).
template <typename T, int NJ>
__global__ void __launch_bounds__(kThr)
    k_delta_seq_bwd(const T *__restrict__ dy, const float *__restrict__ dh_final, const T *__restrict__ g,
                    const T *__restrict__ beta, const T *__restrict__ Bm, const T *__restrict__ Cm, int64_t L, int H, int P,
                    int G, int N, T *__restrict__ dx, float *__restrict__ z_out, float *__restrict__ seg_cot,
                    float *__restrict__ dh0) {
    __shared__ float ks[kTb * NJ * 32], qs[kTb * NJ * 32], ys[kTb * kWarps * kRows], as[kTb], bs[kTb];
    const int h = blockIdx.y, b = blockIdx.z, grp = h / (H / G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pc = blockIdx.x * kWarps * kRows, p0 = pc + warp * kRows;
    const int64_t row0 = ((int64_t)b * H + h) * P, ns = (L + kSeg - 1) / kSeg;
    float s[kRows][NJ];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = lane + 32 * j;
            s[r][j] = dh_final && p0 + r < P && n < N ? dh_final[(row0 + p0 + r) * N + n] : 0.f;
        }
    for (int64_t t0 = (L - 1) / kTb * kTb; t0 >= 0; t0 -= kTb) {
        __syncthreads();
        stage_rows<T, NJ>(Bm, L, t0, G, N, b, grp, ks);
        stage_rows<T, NJ>(Cm, L, t0, G, N, b, grp, qs);
        for (int i = tid; i < kTb * kWarps * kRows; i += kThr) {
            const int t = i / (kWarps * kRows), p = pc + i % (kWarps * kRows);
            ys[i] = t0 + t < L && p < P ? to_f32(dy[(((int64_t)b * L + t0 + t) * H + h) * P + p]) : 0.f;
        }
        if (tid < kTb && t0 + tid < L) {
            as[tid] = expf(to_f32(g[((int64_t)b * L + t0 + tid) * H + h]));
            bs[tid] = to_f32(beta[((int64_t)b * L + t0 + tid) * H + h]);
        }
        __syncthreads();
        for (int t = (L - t0 < kTb ? (int)(L - t0) : kTb) - 1; t >= 0; --t) {
            const int64_t tt = t0 + t;
            if (tt == L - 1 || (tt + 1) % kSeg == 0) {
                const int64_t c = tt / kSeg;
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int n = lane + 32 * j;
                        if (p0 + r < P && n < N)
                            seg_cot[((((int64_t)b * H + h) * ns + c) * P + p0 + r) * N + n] = s[r][j];
                    }
            }
            const float a = as[t], bt = bs[t];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float d = ys[t * kWarps * kRows + warp * kRows + r];
                float pk = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    s[r][j] = fmaf(d, qs[t * NJ * 32 + lane + 32 * j], s[r][j]);
                    pk = fmaf(s[r][j], ks[t * NJ * 32 + lane + 32 * j], pk);
                }
                const float z = warp_sum(pk), dv = bt * z;
#pragma unroll
                for (int j = 0; j < NJ; ++j) s[r][j] = a * fmaf(-dv, ks[t * NJ * 32 + lane + 32 * j], s[r][j]);
                const int64_t at = (((int64_t)b * L + tt) * H + h) * P + p0 + r;
                if (lane == 0 && p0 + r < P) {
                    store_as(dx + at, dv);
                    z_out[at] = z;
                }
            }
        }
    }
    if (dh0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = lane + 32 * j;
                if (p0 + r < P && n < N) dh0[(row0 + p0 + r) * N + n] = s[r][j];
            }
    }
}

// One segment of one head: grid (segments, H, B). With S the entering state, D the leaving cotangent,
// cum the cumulated log decay within the segment and E_ij = exp(cum_i - cum_j) for i >= j:
//   dP_ij = (dy_i.u_j) E_ij (i >= j),  dM_ij = -(r_i.u_j) E_ij (i > j),  u = beta err, r = beta z,
//   dC_i = exp(cum_i) dy_i S + sum_j dP_ij k_j,
//   dB_i = sum_j dP_ji q_j + (dM_ij + dM_ji) k_j + exp(cum_end - cum_i) u_i D - exp(cum_i) r_i S,
//   dbeta_i = z_i.err_i, and dg the reverse cumulative sum of the derivative with respect to cum.
// A thread owns one column n for all tokens; dy, u and r stand transposed in shared memory, so that
// four tokens' values come with one 16-byte broadcast.
constexpr int kTp = kSeg + 4;  // padded token stride of the transposed arrays (16-byte rows)

template <typename T>
__global__ void __launch_bounds__(kThr)
    k_delta_grads(const T *__restrict__ dy, const T *__restrict__ g, const T *__restrict__ beta, const T *__restrict__ Bm,
                  const T *__restrict__ Cm, const float *__restrict__ seg_states, const float *__restrict__ seg_cot,
                  const float *__restrict__ err, const float *__restrict__ zz, int64_t L, int H, int P, int G, int N,
                  float *__restrict__ dB_part, float *__restrict__ dC_part, T *__restrict__ dg, T *__restrict__ dbeta) {
    extern __shared__ __align__(16) float sm[];
    const int N1 = N | 1;
    float *dyT = sm;                      // [P][kTp]
    float *uT = dyT + P * kTp;            // [P][kTp]
    float *rT = uT + P * kTp;             // [P][kTp]
    float *ks = rT + P * kTp;             // [kSeg][N1]
    float *qs = ks + kSeg * N1;           // [kSeg][N1]
    float *wP = qs + kSeg * N1;           // [kSeg][33]
    float *wM = wP + kSeg * 33;           // [kSeg][33], dM + dM^T
    float *pair = wM + kSeg * 33;         // [kSeg][33]
    float *dots = pair + kSeg * 33;       // [kWarps][kSeg]
    float *tail = dots + kWarps * kSeg;   // [kWarps]
    float *eg = tail + kWarps;            // [kSeg]
    float *ek = eg + kSeg;                // [kSeg]
    float *bt = ek + kSeg;                // [kSeg]
    float *zd = bt + kSeg;                // [kSeg]
    __shared__ double cum[kSeg];
    const int64_t c = blockIdx.x, ns = gridDim.x, t0 = c * kSeg;
    const int h = blockIdx.y, b = blockIdx.z, grp = h / (H / G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nt = L - t0 < kSeg ? (int)(L - t0) : kSeg;
    if (tid == 0) {
        double acc = 0.0;
        for (int t = 0; t < kSeg; ++t) {
            if (t < nt) acc += clamp_log_decay(to_f32(g[((int64_t)b * L + t0 + t) * H + h]));
            cum[t] = acc;
        }
    }
    if (tid < kSeg) bt[tid] = tid < nt ? to_f32(beta[((int64_t)b * L + t0 + tid) * H + h]) : 0.f;
    for (int i = tid; i < kSeg * N; i += kThr) {
        const int t = i / N, n = i % N;
        const int64_t at = (((int64_t)b * L + t0 + t) * G + grp) * N + n;
        ks[t * N1 + n] = t < nt ? to_f32(Bm[at]) : 0.f;
        qs[t * N1 + n] = t < nt ? to_f32(Cm[at]) : 0.f;
    }
    __syncthreads();
    if (tid < kSeg) {
        eg[tid] = expf((float)cum[tid]);
        ek[tid] = expf((float)(cum[kSeg - 1] - cum[tid]));
    }
    for (int t = warp; t < kSeg; t += kWarps) {  // a warp per token: also z.err
        float d = 0.f;
        for (int p = lane; p < P; p += 32) {
            const int64_t at = (((int64_t)b * L + t0 + t) * H + h) * P + p;
            const float ev = t < nt ? err[at] : 0.f, zv = t < nt ? zz[at] : 0.f;
            dyT[p * kTp + t] = t < nt ? to_f32(dy[at]) : 0.f;
            uT[p * kTp + t] = bt[t] * ev;
            rT[p * kTp + t] = bt[t] * zv;
            d = fmaf(zv, ev, d);
        }
        d = warp_sum(d);
        if (lane == 0) zd[t] = d;
    }
    __syncthreads();
    if (tid < nt) store_as(dbeta + ((int64_t)b * L + t0 + tid) * H + h, zd[tid]);
    for (int i = warp; i < kSeg; i += kWarps) {
        const int j = lane;
        float dp = 0.f, dm = 0.f, qk = 0.f, kk = 0.f;
        if (j <= i) {
            for (int p = 0; p < P; ++p) {
                dp = fmaf(dyT[p * kTp + i], uT[p * kTp + j], dp);
                dm = fmaf(rT[p * kTp + i], uT[p * kTp + j], dm);
            }
            for (int n = 0; n < N; ++n) {
                qk = fmaf(qs[i * N1 + n], ks[j * N1 + n], qk);
                kk = fmaf(ks[i * N1 + n], ks[j * N1 + n], kk);
            }
            const float e = expf((float)(cum[i] - cum[j]));
            dp *= e;
            dm = j < i ? -dm * e : 0.f;
        }
        wP[i * 33 + j] = j <= i ? dp : 0.f;
        pair[i * 33 + j] = j <= i ? dp * qk + dm * kk : 0.f;
        if (j < i) wM[i * 33 + j] = wM[j * 33 + i] = dm;
        if (j == i) wM[i * 33 + i] = 0.f;
    }
    const float *S = seg_states + (((int64_t)b * H + h) * ns + c) * P * N;
    const float *D = seg_cot + (((int64_t)b * H + h) * ns + c) * P * N;
    const int n = tid;
    float fq[kSeg], fk[kSeg], fu[kSeg], ds = 0.f;
#pragma unroll
    for (int t = 0; t < kSeg; ++t) fq[t] = fk[t] = fu[t] = 0.f;
    if (n < N) {
        for (int p = 0; p < P; ++p) {
            const float sv = S[(int64_t)p * N + n], dv = D[(int64_t)p * N + n];
            ds = fmaf(sv, dv, ds);
#pragma unroll
            for (int t = 0; t < kSeg; t += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(dyT + p * kTp + t);
                const float4 r = *reinterpret_cast<const float4 *>(rT + p * kTp + t);
                const float4 u = *reinterpret_cast<const float4 *>(uT + p * kTp + t);
                fq[t] = fmaf(a.x, sv, fq[t]), fq[t + 1] = fmaf(a.y, sv, fq[t + 1]);
                fq[t + 2] = fmaf(a.z, sv, fq[t + 2]), fq[t + 3] = fmaf(a.w, sv, fq[t + 3]);
                fk[t] = fmaf(r.x, sv, fk[t]), fk[t + 1] = fmaf(r.y, sv, fk[t + 1]);
                fk[t + 2] = fmaf(r.z, sv, fk[t + 2]), fk[t + 3] = fmaf(r.w, sv, fk[t + 3]);
                fu[t] = fmaf(u.x, dv, fu[t]), fu[t + 1] = fmaf(u.y, dv, fu[t + 1]);
                fu[t + 2] = fmaf(u.z, dv, fu[t + 2]), fu[t + 3] = fmaf(u.w, dv, fu[t + 3]);
            }
        }
    }
    // the derivative with respect to cum: per token in `dots`, the end's share in `tail`
    float end = expf((float)cum[kSeg - 1]) * ds;
#pragma unroll
    for (int t = 0; t < kSeg; ++t) {
        const float kn = n < N ? ks[t * N1 + n] : 0.f, qn = n < N ? qs[t * N1 + n] : 0.f;
        fq[t] *= eg[t];
        fu[t] *= ek[t];
        const float U = fu[t] * kn;
        end += U;
        const float d = warp_sum(fq[t] * qn - eg[t] * fk[t] * kn - U);
        if (lane == 0) dots[warp * kSeg + t] = d;
        fk[t] = fu[t] - eg[t] * fk[t];
    }
    end = warp_sum(end);
    if (lane == 0) tail[warp] = end;
    __syncthreads();
    if (n < N) {
        for (int j = 0; j < kSeg; ++j) {
            const float kn = ks[j * N1 + n], qn = qs[j * N1 + n];
#pragma unroll
            for (int t = 0; t < kSeg; ++t) {
                fq[t] = fmaf(wP[t * 33 + j], kn, fq[t]);
                fk[t] = fmaf(wP[j * 33 + t], qn, fk[t]);
                fk[t] = fmaf(wM[j * 33 + t], kn, fk[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < kSeg; ++t) {
            if (t < nt) {
                const int64_t at = (((int64_t)b * L + t0 + t) * H + h) * N + n;
                dC_part[at] = fq[t];
                dB_part[at] = fk[t];
            }
        }
    }
    if (warp == 0) {
        const int i = lane;
        float d = 0.f;
        for (int w = 0; w < kWarps; ++w) d += dots[w * kSeg + i];
        for (int j = 0; j < kSeg; ++j) d += pair[i * 33 + j] - pair[j * 33 + i];
        if (i == kSeg - 1)
            for (int w = 0; w < kWarps; ++w) d += tail[w];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {  // sum over the tokens from i to the end
            const float up = __shfl_down_sync(0xffffffffu, d, o);
            if (i + o < 32) d += up;
        }
        if (i < nt) store_as(dg + ((int64_t)b * L + t0 + i) * H + h, d);
    }
}

// Sums over the heads of each group, in head order. One thread per output element.
template <typename T>
__global__ void k_delta_group_sum(const float *__restrict__ dB_part, const float *__restrict__ dC_part, int64_t tokens,
                                  int H, int G, int N, T *__restrict__ dBm, T *__restrict__ dCm) {
    const int64_t total = tokens * G * N;
    const int per = H / G;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int n = (int)(i % N), g = (int)(i / N % G);
        const int64_t t = i / N / G;
        float sb = 0.f, sc = 0.f;
        for (int h = g * per; h < (g + 1) * per; ++h) {
            sb += dB_part[(t * H + h) * N + n];
            sc += dC_part[(t * H + h) * N + n];
        }
        store_as(dBm + i, sb);
        store_as(dCm + i, sc);
    }
}

// One token: grid (ceil(P / kStepRows), H, B), 8 warps, 4 rows per warp whose loads are issued
// together. state_out may be state_in: a row is whole in registers before it is written, and only
// its own warp touches it (so neither carries __restrict__). N % 4 == 0.
constexpr int kStepPer = 4, kStepRows = kWarps * kStepPer;

template <typename T, int NV>
__global__ void __launch_bounds__(kThr)
    k_delta_step(const float *state_in, float *state_out, const T *__restrict__ x, const T *__restrict__ g,
                 const T *__restrict__ beta, const T *__restrict__ Bm, const T *__restrict__ Cm, int H, int P, int G, int N,
                 T *__restrict__ y) {
    const int h = blockIdx.y, b = blockIdx.z, grp = h / (H / G);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int p0 = blockIdx.x * kStepRows + warp * kStepPer;
    if (p0 >= P) return;
    const int64_t row0 = ((int64_t)b * H + h) * P + p0;
    const int nv = N / 4;
    float4 s[kStepPer][NV];
#pragma unroll
    for (int r = 0; r < kStepPer; ++r)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = lane + 32 * j;
            s[r][j] = v < nv && p0 + r < P ? reinterpret_cast<const float4 *>(state_in + (row0 + r) * N)[v]
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    float k[NV][4], q[NV][4], kq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = lane + 32 * j;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t at = ((int64_t)b * G + grp) * N + 4 * v + e;
            k[j][e] = v < nv ? to_f32(Bm[at]) : 0.f;
            q[j][e] = v < nv ? to_f32(Cm[at]) : 0.f;
            kq = fmaf(k[j][e], q[j][e], kq);
        }
    }
    const float a = expf(to_f32(g[(int64_t)b * H + h])), bt = to_f32(beta[(int64_t)b * H + h]);
    kq = warp_sum(kq);
#pragma unroll
    for (int r = 0; r < kStepPer; ++r) {
        float pk = 0.f, pq = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            pk = fmaf(s[r][j].x, k[j][0], fmaf(s[r][j].y, k[j][1], fmaf(s[r][j].z, k[j][2], fmaf(s[r][j].w, k[j][3], pk))));
            pq = fmaf(s[r][j].x, q[j][0], fmaf(s[r][j].y, q[j][1], fmaf(s[r][j].z, q[j][2], fmaf(s[r][j].w, q[j][3], pq))));
        }
        pk = warp_sum(pk);
        pq = warp_sum(pq);
        if (p0 + r < P) {
            const float u = bt * (to_f32(x[row0 + r]) - a * pk);
            float4 *dst = reinterpret_cast<float4 *>(state_out + (row0 + r) * N);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int v = lane + 32 * j;
                float4 o;
                o.x = fmaf(a, s[r][j].x, u * k[j][0]);
                o.y = fmaf(a, s[r][j].y, u * k[j][1]);
                o.z = fmaf(a, s[r][j].z, u * k[j][2]);
                o.w = fmaf(a, s[r][j].w, u * k[j][3]);
                if (v < nv) dst[v] = o;
            }
            if (lane == 0) store_as(y + row0 + r, fmaf(a, pq, u * kq));
        }
    }
}

template <typename T, int NJ>
cudaError_t seq_launch(const DeltaProblem &p, float *seg_states, float *err, cudaStream_t s) {
    dim3 grid((unsigned)((p.P + kWarps * kRows - 1) / (kWarps * kRows)), (unsigned)p.H, (unsigned)p.B);
    k_delta_seq<T, NJ><<<grid, kThr, 0, s>>>(static_cast<const T *>(p.x), static_cast<const T *>(p.g),
                                             static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
                                             p.y ? static_cast<const T *>(p.Cm) : nullptr, p.h0, p.L, (int)p.H, (int)p.P,
                                             (int)p.G, (int)p.N, static_cast<T *>(p.y), p.h_final, seg_states, err);
    return cudaGetLastError();
}

template <typename T>
cudaError_t seq_typed(const DeltaProblem &p, float *seg_states, float *err, cudaStream_t s) {
    if (p.N <= 32) return seq_launch<T, 1>(p, seg_states, err, s);
    if (p.N <= 64) return seq_launch<T, 2>(p, seg_states, err, s);
    if (p.N <= 128) return seq_launch<T, 4>(p, seg_states, err, s);
    return seq_launch<T, 8>(p, seg_states, err, s);
}

template <typename T, int NJ>
cudaError_t seq_bwd_launch(const DeltaProblem &p, const DeltaGrads &gr, float *z, float *seg_cot, cudaStream_t s) {
    dim3 grid((unsigned)((p.P + kWarps * kRows - 1) / (kWarps * kRows)), (unsigned)p.H, (unsigned)p.B);
    k_delta_seq_bwd<T, NJ><<<grid, kThr, 0, s>>>(static_cast<const T *>(gr.dy), gr.dh_final, static_cast<const T *>(p.g),
                                                 static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
                                                 static_cast<const T *>(p.Cm), p.L, (int)p.H, (int)p.P, (int)p.G, (int)p.N,
                                                 static_cast<T *>(gr.dx), z, seg_cot, gr.dh0);
    return cudaGetLastError();
}

size_t grads_smem(const DeltaProblem &p) {
    return sizeof(float) * (size_t)(3 * p.P * kTp + 2 * kSeg * (p.N | 1) + 3 * kSeg * 33 + kWarps * kSeg + kWarps + 4 * kSeg);
}

// Workspace of the general backward, as byte offsets.
struct BwdLayout {
    size_t states, cot, err, z, dB, dC, total;
};
BwdLayout bwd_layout(const DeltaProblem &p) {
    const size_t ns = (size_t)((p.L + kSeg - 1) / kSeg), seg = (size_t)(p.B * p.H) * ns * (size_t)(p.P * p.N) * 4;
    const size_t rows = (size_t)(p.B * p.L * p.H * p.P) * 4, cols = (size_t)(p.B * p.L * p.H * p.N) * 4;
    BwdLayout l{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, kWsAlign);
        return here;
    };
    l.states = take(seg);
    l.cot = take(seg);
    l.err = take(rows);
    l.z = take(rows);
    l.dB = take(cols);
    l.dC = take(cols);
    l.total = at;
    return l;
}

template <typename T>
cudaError_t bwd_typed(const DeltaProblem &p, const DeltaGrads &gr, void *ws, cudaStream_t s) {
    const BwdLayout l = bwd_layout(p);
    char *base = static_cast<char *>(ws);
    float *states = reinterpret_cast<float *>(base + l.states), *cot = reinterpret_cast<float *>(base + l.cot);
    float *err = reinterpret_cast<float *>(base + l.err), *z = reinterpret_cast<float *>(base + l.z);
    float *dB = reinterpret_cast<float *>(base + l.dB), *dC = reinterpret_cast<float *>(base + l.dC);
    DeltaProblem f = p;  // the states alone: no output, no final state
    f.y = nullptr;
    f.h_final = nullptr;
    cudaError_t e = seq_typed<T>(f, states, err, s);
    if (e) return e;
    if (p.N <= 32) e = seq_bwd_launch<T, 1>(p, gr, z, cot, s);
    else if (p.N <= 64) e = seq_bwd_launch<T, 2>(p, gr, z, cot, s);
    else if (p.N <= 128) e = seq_bwd_launch<T, 4>(p, gr, z, cot, s);
    else e = seq_bwd_launch<T, 8>(p, gr, z, cot, s);
    if (e) return e;
    const size_t smem = grads_smem(p);
    if ((e = cudaFuncSetAttribute(k_delta_grads<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem))) return e;
    dim3 grid((unsigned)((p.L + kSeg - 1) / kSeg), (unsigned)p.H, (unsigned)p.B);
    k_delta_grads<T><<<grid, kThr, smem, s>>>(static_cast<const T *>(gr.dy), static_cast<const T *>(p.g),
                                              static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
                                              static_cast<const T *>(p.Cm), states, cot, err, z, p.L, (int)p.H, (int)p.P,
                                              (int)p.G, (int)p.N, dB, dC, static_cast<T *>(gr.dg),
                                              static_cast<T *>(gr.dbeta));
    if ((e = cudaGetLastError())) return e;
    return delta_group_sum_launch(p, dB, dC, gr.dBm, gr.dCm, s);
}

template <typename T, int NV>
void step_launch(const DeltaProblem &p, const float *in, float *out, cudaStream_t s) {
    dim3 grid((unsigned)((p.P + kStepRows - 1) / kStepRows), (unsigned)p.H, (unsigned)p.B);
    k_delta_step<T, NV><<<grid, kThr, 0, s>>>(in, out, static_cast<const T *>(p.x), static_cast<const T *>(p.g),
                                              static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
                                              static_cast<const T *>(p.Cm), (int)p.H, (int)p.P, (int)p.G, (int)p.N,
                                              static_cast<T *>(p.y));
}

}  // namespace

cudaError_t delta_group_sum_launch(const DeltaProblem &p, const float *dB_part, const float *dC_part, void *dBm, void *dCm,
                                   cudaStream_t s) {
    const int64_t total = p.B * p.L * p.G * p.N, blocks = (total + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 148 * 16 ? blocks : 148 * 16);
    if (p.dtype == SSD_F32)
        k_delta_group_sum<float><<<grid, 256, 0, s>>>(dB_part, dC_part, p.B * p.L, (int)p.H, (int)p.G, (int)p.N,
                                                      static_cast<float *>(dBm), static_cast<float *>(dCm));
    else
        k_delta_group_sum<__nv_bfloat16><<<grid, 256, 0, s>>>(dB_part, dC_part, p.B * p.L, (int)p.H, (int)p.G, (int)p.N,
                                                              static_cast<__nv_bfloat16 *>(dBm),
                                                              static_cast<__nv_bfloat16 *>(dCm));
    return cudaGetLastError();
}

cudaError_t delta_seq_fwd(const DeltaProblem &p, cudaStream_t s) {
    return p.dtype == SSD_F32 ? seq_typed<float>(p, nullptr, nullptr, s) : seq_typed<__nv_bfloat16>(p, nullptr, nullptr, s);
}

size_t delta_seq_bwd_workspace_bytes(const DeltaProblem &p) { return bwd_layout(p).total; }

cudaError_t delta_seq_bwd(const DeltaProblem &p, const DeltaGrads &g, void *ws, cudaStream_t s) {
    return p.dtype == SSD_F32 ? bwd_typed<float>(p, g, ws, s) : bwd_typed<__nv_bfloat16>(p, g, ws, s);
}

cudaError_t delta_step(const DeltaProblem &p, const float *state_in, float *state_out, cudaStream_t s) {
    if (p.dtype == SSD_F32) {
        if (p.N <= 128) step_launch<float, 1>(p, state_in, state_out, s);
        else step_launch<float, 2>(p, state_in, state_out, s);
    } else {
        if (p.N <= 128) step_launch<__nv_bfloat16, 1>(p, state_in, state_out, s);
        else step_launch<__nv_bfloat16, 2>(p, state_in, state_out, s);
    }
    return cudaGetLastError();
}

}  // namespace ssd
