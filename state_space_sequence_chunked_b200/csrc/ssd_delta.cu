// The gated delta rule: its general path (any headdim, dstate <= 256, fp32 and bf16) and the
// one-token step. Per (b, h), with group k = B_t, q = C_t and a_t = exp(g_t):
//     h' = a_t h_{t-1},  err_t = x_t - h' k_t,  u_t = beta_t err_t,  h_t = h' + u_t k_t^T,  y_t = h_t q_t.
// The rows p of the state are independent given k and q: a row is h_t[p, :] = a_t h[p, :] + u_t[p] k_t,
// so a warp keeps whole rows in registers and nothing crosses warps.
//
//   k_delta_seq       four tokens at a time, a row in 8 lanes. All dot products of the four, h k_i and h q_i,
//                     are of the state before them; what tokens j < i of the four add is a
//                     combination of the products k_j.k_i and k_j.q_i, which the staging warps
//                     form beside: one reduction and one update of the state per four tokens. For the
//                     backward pass it also leaves err and the state entering each segment of kSeg.
//   k_delta_seq_bwd   the same walk in reverse: with D the cotangent of h_t,
//                     D += dy_t q_t^T, z_t = D k_t, dx_t = beta_t z_t, D <- a_t (D - dx_t k_t^T).
//                     It needs no state; it leaves z and the cotangent leaving each segment.
//   k_delta_grads     per segment, everything that sums over the rows of the state (dB, dC, dg,
//                     dbeta), from the segment's entering state, leaving cotangent, err and z.
//   k_delta_step      one token, HBM-bound: the state is read and written once.
//
// This is the exact path (fp32 throughout), bound by the latency of its chain and not by a unit: 2 x 777 fp32
// tokens of 6 heads of 40 x 36 take 96 us, 0.12 us a token (token by token with a row in 32 lanes 335 us; two
// rows per lane 141); 37 bf16 tokens of 24 heads of 64 x 128 take 13 us (24 on the tensor cores). bf16 inputs of the
// usual sizes and lengths take the chunked tensor-core path in ssd_delta_mma.cu.
//
// k_delta_step is bound by HBM: 64 sequences of 32 heads of 128 x 128, 51 us, 82% of the measured 6.45 TB/s.
#include <type_traits>

#include "ssd_delta.cuh"

namespace ssd {
namespace {

constexpr int kThr = 256, kWarps = kThr / 32;
constexpr int kSeqRows = 16;  // state rows per CTA of the sequential kernels
constexpr int kSeqWalk = kSeqRows * 8, kSeqThr = kSeqWalk + 128;  // threads that walk, and with those that stage

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Tokens of the sequential kernels in shared memory, as fp32, a block of 4 at a time with the products of its
// keys and queries. Past L: zeros, a = 1, beta = 0 (such a token leaves the state as it is).
template <int NJ>
struct SeqStage {
    static constexpr int tb = NJ < 8 ? 16 : 8, cols = 32 * NJ;
    float4 k[tb * cols / 4], q[tb * cols / 4];
    float x[kSeqRows][tb];      // of the rows: x, or dy
    float a[tb], beta[tb];
    float qk[tb / 4][4][4];     // q_i.k_j, j <= i
    float kk[tb / 4][8];        // k_i.k_j, j < i: (1,0) (2,0) (2,1) (3,0) (3,1) (3,2)
};

// Four warps stage tokens: those after the next ones are on their way in registers while the next ones are written.
// `rows` is x or dy.
template <typename T, int NJ>
struct SeqLoad {
    using S = SeqStage<NJ>;
    static constexpr int kM = S::tb * S::cols / 128, kX = S::tb * kSeqRows / 128;
    T k[kM], q[kM], x[kX], gv, bv;
    __device__ __forceinline__ void fetch(const T *__restrict__ rows, const T *__restrict__ g, const T *__restrict__ beta,
                                          const T *__restrict__ Bm, const T *__restrict__ Cm, int64_t L, int64_t t0, int H, int P,
                                          int G, int N, int b, int h, int pc, int tid) {
        const T zero = T(0.f);
        const int64_t base = (((int64_t)b * L + t0) * G + h / (H / G)) * N;
        const int left = L - t0 < S::tb ? (int)(L - t0) : S::tb;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const int i = tid + 128 * m, t = i / S::cols, n = i % S::cols;
            const bool in = n < N && t < left;
            const int64_t at = in ? base + (int64_t)t * G * N + n : 0;
            k[m] = in ? Bm[at] : zero;
            q[m] = in && Cm ? Cm[at] : zero;
        }
#pragma unroll
        for (int m = 0; m < kX; ++m) {
            const int i = tid + 128 * m, t = i / kSeqRows, r = i % kSeqRows;
            x[m] = t < left && pc + r < P ? rows[(((int64_t)b * L + t0 + t) * H + h) * P + pc + r] : zero;
        }
        const int64_t at = ((int64_t)b * L + t0 + tid) * H + h;
        gv = tid < left ? g[at] : zero;
        bv = tid < left ? beta[at] : zero;
    }
    __device__ __forceinline__ void put(S &st, int tid) const {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            reinterpret_cast<float *>(st.k)[tid + 128 * m] = to_f32(k[m]);
            reinterpret_cast<float *>(st.q)[tid + 128 * m] = to_f32(q[m]);
        }
#pragma unroll
        for (int m = 0; m < kX; ++m) st.x[(tid + 128 * m) % kSeqRows][(tid + 128 * m) / kSeqRows] = to_f32(x[m]);
        if (tid < S::tb) st.a[tid] = expf(to_f32(gv)), st.beta[tid] = to_f32(bv);
    }
};
// What of a block's tokens meets: all by the staging warps, after their writes.
template <int NJ>
__device__ __forceinline__ void seq_pairs(SeqStage<NJ> &st, int tid) {
    using S = SeqStage<NJ>;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    // 10 + 6 products of a block, 8 lanes each
    const int item = tid >> 3, l8 = tid & 7, m = item < 10 ? item : item - 10;
    const int r = (m >= 1) + (m >= 3) + (m >= 6), j = m - r * (r + 1) / 2, i = item < 10 ? r : r + 1;
    const float4 *left = item < 10 ? st.q : st.k;
#pragma unroll
    for (int blk = 0; blk < S::tb / 4; ++blk) {
        float d = 0.f;
#pragma unroll
        for (int v = 0; v < NJ; ++v) {
            const float4 f = left[(4 * blk + i) * (S::cols / 4) + 8 * v + l8], w = st.k[(4 * blk + j) * (S::cols / 4) + 8 * v + l8];
            d = fmaf(f.x, w.x, fmaf(f.y, w.y, fmaf(f.z, w.z, fmaf(f.w, w.w, d))));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (l8 == 0) (item < 10 ? st.qk[blk][i][j] : st.kk[blk][m]) = d;
    }
}

// Staging and walking warps meet here once per stage, each from its own loop.
__device__ __forceinline__ void seq_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kSeqThr) : "memory"); }

// A row of the state, 4 NJ columns per lane: columns 32 v + 4 l8 ..
template <int NJ>
__device__ __forceinline__ void row_load(float2 (&s)[NJ][2], const float *src, bool live, int l8, int N) {
#pragma unroll
    for (int v = 0; v < NJ; ++v) {
        const int n = 32 * v + 4 * l8;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            s[v][e] = make_float2(live && n + 2 * e < N ? src[n + 2 * e] : 0.f, live && n + 2 * e + 1 < N ? src[n + 2 * e + 1] : 0.f);
    }
}
template <int NJ>
__device__ __forceinline__ void row_store(const float2 (&s)[NJ][2], float *dst, int l8, int N) {
#pragma unroll
    for (int v = 0; v < NJ; ++v) {
        const int n = 32 * v + 4 * l8;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (n + 2 * e < N) dst[n + 2 * e] = s[v][e].x;
            if (n + 2 * e + 1 < N) dst[n + 2 * e + 1] = s[v][e].y;
        }
    }
}
__device__ __forceinline__ float2 low2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 high2(float4 v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <int NJ>
__device__ __forceinline__ float row_dot(const float2 (&s)[NJ][2], const float4 *w, int l8) {
    float2 d0 = both(0.f), d1 = d0;
#pragma unroll
    for (int v = 0; v < NJ; ++v) {
        const float4 f = w[8 * v + l8];
        d0 = fma2(s[v][0], low2(f), d0);
        d1 = fma2(s[v][1], high2(f), d1);
    }
    return (d0.x + d1.x) + (d0.y + d1.y);
}
template <int NJ>
__device__ __forceinline__ void row_add(float2 (&s)[NJ][2], float c, const float4 *w, int l8) {
#pragma unroll
    for (int v = 0; v < NJ; ++v) {
        const float4 f = w[8 * v + l8];
        s[v][0] = fma2(both(c), low2(f), s[v][0]);
        s[v][1] = fma2(both(c), high2(f), s[v][1]);
    }
}
template <int NJ>
__device__ __forceinline__ void row_scale(float2 (&s)[NJ][2], float c) {
#pragma unroll
    for (int v = 0; v < NJ; ++v) s[v][0] = mul2(both(c), s[v][0]), s[v][1] = mul2(both(c), s[v][1]);
}
// Eight values per lane, each to be summed over eight neighbouring lanes: halves are exchanged, so that lane l
// ends with the sum of value l.
__device__ __forceinline__ float sums8(float (&v)[8], int lane) {
    int x = 4;
#pragma unroll
    for (int w = 4; w >= 1; w >>= 1, x >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const bool up = lane & x;
            const float send = up ? v[j] : v[j + w], keep = up ? v[j + w] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, x);
        }
    return v[0];
}

// grid (ceil(P / 16), H, B), 4 warps that walk the tokens (a row in 8 lanes) and 4 that stage the next ones.
template <typename T, int NJ, bool kY>
__global__ void __launch_bounds__(kSeqThr, NJ < 8 ? 2 : 1)
    k_delta_seq(const T *__restrict__ x, const T *__restrict__ g, const T *__restrict__ beta, const T *__restrict__ Bm,
                const T *__restrict__ Cm, const float *__restrict__ h0, int64_t L, int H, int P, int G, int N,
                T *__restrict__ y, float *__restrict__ h_final, float *__restrict__ seg_states,
                float *__restrict__ err_out) {
    using S = SeqStage<NJ>;
    __shared__ S st[2];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l8 = lane & 7;
    const int pc = blockIdx.x * kSeqRows, r = warp * 4 + (lane >> 3), p = pc + r;
    const bool live = p < P;
    
    const int64_t row = ((int64_t)b * H + h) * P + p, ns = (L + kSeg - 1) / kSeg;
    if (tid >= kSeqWalk) {
        SeqLoad<T, NJ> in;
        const auto fetch = [&](int64_t t0) { in.fetch(x, g, beta, Bm, Cm, L, t0, H, P, G, N, b, h, pc, tid - kSeqWalk); };
        fetch(0);
        for (int64_t t0 = 0; t0 < L; t0 += S::tb) {
            in.put(st[t0 / S::tb & 1], tid - kSeqWalk);
            if (t0 + S::tb < L) fetch(t0 + S::tb);
            seq_pairs<NJ>(st[t0 / S::tb & 1], tid - kSeqWalk);
            seq_sync();  // these tokens are there, and the others' place is free
        }
        return;
    }
    float2 s[NJ][2];
    row_load<NJ>(s, h0 + row * N, h0 && live, l8, N);
    for (int64_t t0 = 0; t0 < L; t0 += S::tb) {
        const S &c = st[t0 / S::tb & 1];
        seq_sync();
        for (int blk = 0; blk < S::tb / 4 && t0 + 4 * blk < L; ++blk) {
            const int64_t t = t0 + 4 * blk;
            if (seg_states && t % kSeg == 0 && live)
                row_store<NJ>(s, seg_states + ((((int64_t)b * H + h) * ns + t / kSeg) * P + p) * N, l8, N);
            const float4 *k = c.k + blk * S::cols, *q = c.q + blk * S::cols;
            float d[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = row_dot<NJ>(s, k + i * (S::cols / 4), l8);
                d[4 + i] = kY ? row_dot<NJ>(s, q + i * (S::cols / 4), l8) : 0.f;
            }
            const float own = sums8(d, lane);  // h.k of token l8, or h.q of token l8 - 4
            const float4 a4 = *reinterpret_cast<const float4 *>(&c.a[4 * blk]), b4 = *reinterpret_cast<const float4 *>(&c.beta[4 * blk]);
            const float a[4] = {a4.x, a4.y, a4.z, a4.w}, bt[4] = {b4.x, b4.y, b4.z, b4.w};
            const float4 m0 = *reinterpret_cast<const float4 *>(&c.kk[blk][0]), m1 = *reinterpret_cast<const float4 *>(&c.kk[blk][4]);
            const float kk[6] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y};
            const float4 qr = *reinterpret_cast<const float4 *>(&c.qk[blk][l8 & 3][0]);
            const float qk[4] = {qr.x, qr.y, qr.z, qr.w};
            const float4 x4 = *reinterpret_cast<const float4 *>(&c.x[r][4 * blk]);
            const float xv[4] = {x4.x, x4.y, x4.z, x4.w};
            float u[4], err[4], yv = own;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // h' k_i: the block's earlier tokens by their keys' products
                float v = __shfl_sync(0xffffffffu, own, (lane & 24) + i);
#pragma unroll
                for (int j = 0; j < i; ++j) v = fmaf(u[j], kk[i * (i - 1) / 2 + j], a[j] * v);
                err[i] = xv[i] - a[i] * v;
                u[i] = bt[i] * err[i];
                const float n = fmaf(u[i], qk[i], a[i] * yv);
                yv = i <= (l8 & 3) ? n : yv;
            }
            const int64_t tt = t + (l8 & 3), at = (((int64_t)b * L + tt) * H + h) * P + p;
            if (live && tt < L) {
                if (l8 >= 4) {
                    if (kY) store_as(y + at, yv);
                } else if (err_out) {
                    err_out[at] = (l8 & 2) ? (l8 & 1 ? err[3] : err[2]) : (l8 & 1 ? err[1] : err[0]);
                }
            }
            const float c2 = a[3], c1 = c2 * a[2], c0 = c1 * a[1], ci[4] = {c0, c1, c2, 1.f};
            row_scale<NJ>(s, c0 * a[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) row_add<NJ>(s, ci[i] * u[i], k + i * (S::cols / 4), l8);
        }
    }
    if (h_final && live) row_store<NJ>(s, h_final + row * N, l8, N);
}

// grid (ceil(P / 16), H, B), warps as above.
template <typename T, int NJ>
__global__ void __launch_bounds__(kSeqThr, NJ < 8 ? 2 : 1)
    k_delta_seq_bwd(const T *__restrict__ dy, const float *__restrict__ dh_final, const T *__restrict__ g,
                    const T *__restrict__ beta, const T *__restrict__ Bm, const T *__restrict__ Cm, int64_t L, int H, int P,
                    int G, int N, T *__restrict__ dx, float *__restrict__ z_out, float *__restrict__ seg_cot,
                    float *__restrict__ dh0) {
    using S = SeqStage<NJ>;
    __shared__ S st[2];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l8 = lane & 7;
    const int pc = blockIdx.x * kSeqRows, r = warp * 4 + (lane >> 3), p = pc + r;
    const bool live = p < P;
    
    const int64_t row = ((int64_t)b * H + h) * P + p, ns = (L + kSeg - 1) / kSeg, first = (L - 1) / S::tb * S::tb;
    if (tid >= kSeqWalk) {
        SeqLoad<T, NJ> in;
        const auto fetch = [&](int64_t t0) { in.fetch(dy, g, beta, Bm, Cm, L, t0, H, P, G, N, b, h, pc, tid - kSeqWalk); };
        fetch(first);
        for (int64_t t0 = first; t0 >= 0; t0 -= S::tb) {
            in.put(st[t0 / S::tb & 1], tid - kSeqWalk);
            if (t0 > 0) fetch(t0 - S::tb);
            seq_pairs<NJ>(st[t0 / S::tb & 1], tid - kSeqWalk);
            seq_sync();
        }
        return;
    }
    float2 s[NJ][2];
    row_load<NJ>(s, dh_final + row * N, dh_final && live, l8, N);
    for (int64_t t0 = first; t0 >= 0; t0 -= S::tb) {
        const S &c = st[t0 / S::tb & 1];
        seq_sync();
        for (int blk = S::tb / 4 - 1; blk >= 0; --blk) {
            const int64_t t = t0 + 4 * blk;
            if (t >= L) continue;
            if ((t + 4 >= L || (t + 4) % kSeg == 0) && live)
                row_store<NJ>(s, seg_cot + ((((int64_t)b * H + h) * ns + t / kSeg) * P + p) * N, l8, N);
            const float4 *k = c.k + blk * S::cols, *q = c.q + blk * S::cols;
            // D k of the four tokens (as eight values; the last four are not used)
            float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = row_dot<NJ>(s, k + i * (S::cols / 4), l8);
            const float own = sums8(d, lane);
            const float4 a4 = *reinterpret_cast<const float4 *>(&c.a[4 * blk]), b4 = *reinterpret_cast<const float4 *>(&c.beta[4 * blk]);
            const float a[4] = {a4.x, a4.y, a4.z, a4.w}, bt[4] = {b4.x, b4.y, b4.z, b4.w};
            const float4 m0 = *reinterpret_cast<const float4 *>(&c.kk[blk][0]), m1 = *reinterpret_cast<const float4 *>(&c.kk[blk][4]);
            const float kk[6] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y};
            const float4 y4 = *reinterpret_cast<const float4 *>(&c.x[r][4 * blk]);
            const float yv[4] = {y4.x, y4.y, y4.z, y4.w};
            float dv[4], zi = 0.f;
#pragma unroll
            for (int i = 3; i >= 0; --i) {  // D k_i: the later tokens of the block by their products with k_i
                float v = __shfl_sync(0xffffffffu, own, (lane & 24) + i);
#pragma unroll
                for (int j = 3; j > i; --j)
                    v = a[j] * fmaf(yv[j], c.qk[blk][j][i], fmaf(-dv[j], kk[j * (j - 1) / 2 + i], v));
                const float z = fmaf(yv[i], c.qk[blk][i][i], v);
                dv[i] = bt[i] * z;
                if (l8 == i) zi = z;
            }
            const float c1 = a[0] * a[1], c2 = c1 * a[2], c3 = c2 * a[3], ci[4] = {a[0], c1, c2, c3};
            row_scale<NJ>(s, c3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                row_add<NJ>(s, ci[i] * yv[i], q + i * (S::cols / 4), l8);
                row_add<NJ>(s, -ci[i] * dv[i], k + i * (S::cols / 4), l8);
            }
            const int64_t at = (((int64_t)b * L + t + l8) * H + h) * P + p;
            if (l8 < 4 && live && t + l8 < L) {
                z_out[at] = zi;
                store_as(dx + at, c.beta[4 * blk + l8] * zi);
            }
        }
    }
    if (dh0 && live) row_store<NJ>(s, dh0 + row * N, l8, N);
}

// One segment of one head: grid (segments, H, B). With S the entering state, D the leaving cotangent,
// cum the cumulated log decay within the segment and E_ij = exp(cum_i - cum_j) for i >= j:
//   dP_ij = (dy_i.u_j) E_ij (i >= j),  dM_ij = -(r_i.u_j) E_ij (i > j),  u = beta err, r = beta z,
//   dC_i = exp(cum_i) dy_i S + sum_j dP_ij k_j,
//   dB_i = sum_j dP_ji q_j + (dM_ij + dM_ji) k_j + exp(cum_end - cum_i) u_i D - exp(cum_i) r_i S,
//   dbeta_i = z_i.err_i, and dg_i the sum of what passes the decay of token i:
//   sum over t >= i > j of dP_tj q_t.k_j + dM_tj k_t.k_j,  sum over t >= i of exp(cum_t) (dy_t.S q_t - r_t.S k_t),
//   sum over t < i of U_t = exp(cum_end - cum_t) u_t.D k_t,  and exp(cum_end) <D, S>.
// No term of these is taken off again (as it is in a cumulative sum of the derivative with respect to cum, where
// the pairs on one side of i come in and go out): dg shrinks with exp(g), and its errors with it.
// The three products with S and D are register tiles: a warp holds TK tokens by all columns (a lane every 32nd) and
// takes them from dy, u and r, transposed in shared memory, four tokens per 16-byte broadcast. Where two warps
// share a tile, each takes a half of the state rows and then a half of the pairs' tokens j; they meet once, at the end.
// Bound by the latency of its loads and by shared memory: 50 heads of 64 x 128, 5 x 305 fp32 tokens, 410 us (452 with
// TK = 8 there, which leaves room for one CTA per SM); 48 heads of 243 x 34, 3602 tokens, 1376 us (a thread per column and
// all tokens 1236 and 6919).
constexpr int kTp = kSeg + 4;  // padded token stride of the transposed arrays (16-byte rows)
// row stride of keys and queries: 4 modulo 32 floats, so that 8 rows' 16-byte vectors fall in different banks
__host__ __device__ constexpr int grads_stride(int N) { return N <= 4 ? 4 : (N - 4 + 31) / 32 * 32 + 4; }

// err or z as the sequential kernels leave them, or in two parts
template <typename T, bool kParts>
struct Row {
    const float *v;
    __device__ __forceinline__ float operator[](int64_t i) const { return __ldg(v + i); }
};
template <typename T>
struct Row<T, true> {
    const T *hi, *lo;
    __device__ __forceinline__ float operator[](int64_t i) const { return to_f32(hi[i]) + to_f32(lo[i]); }
};
template <int NJ>
struct GradsTile {
    static constexpr int TK = NJ >= 4 ? 4 : 8, groups = kSeg / TK, split = kWarps / groups;  // tokens; warps by tokens, by rows
    static constexpr int U = NJ <= 2 ? 8 : 2;  // rows of S and D in flight
};

template <typename T, int NJ, bool kParts>
__global__ void __launch_bounds__(kThr)
    k_delta_grads(const T *__restrict__ dy, const T *__restrict__ g, const T *__restrict__ beta, const T *__restrict__ Bm,
                  const T *__restrict__ Cm, const float *__restrict__ seg_states, const float *__restrict__ seg_cot,
                  const Row<T, kParts> err, const Row<T, kParts> zz, int64_t L, int H, int P, int G, int N,
                  float *__restrict__ dB_part, float *__restrict__ dC_part, T *__restrict__ dg, T *__restrict__ dbeta,
                  T *__restrict__ dx) {
    using Z = GradsTile<NJ>;
    constexpr int TK = Z::TK, PS = Z::split;
    extern __shared__ __align__(16) float sm[];
    const int NP = grads_stride(N);
    float *dyT = sm;                      // [P][kTp]
    float *uT = dyT + P * kTp;            // [P][kTp]
    float *rT = uT + P * kTp;             // [P][kTp]
    float *ks = rT + P * kTp;             // [kSeg][NP]
    float *qs = ks + kSeg * NP;           // [kSeg][NP]
    float *wPt = qs + kSeg * NP;          // [j][kTp]: dP_tj
    float *wP = wPt + kSeg * kTp;         // [j][kTp]: dP_jt
    float *wM = wP + kSeg * kTp;          // [j][kTp]: dM_tj + dM_jt
    float *pair = wM + kSeg * kTp;        // [kSeg][33]
    __shared__ float dots[2][PS][kSeg], ends[kWarps], eg[kSeg], ek[kSeg], bt[kSeg], zd[kSeg];
    __shared__ double cum[kSeg];
    const int64_t c = blockIdx.x, ns = gridDim.x, t0 = c * kSeg;
    const int h = blockIdx.y, b = blockIdx.z, grp = h / (H / G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nt = L - t0 < kSeg ? (int)(L - t0) : kSeg;
    if (warp == 0) {  // cumulated log decay, a token per lane
        double sum = lane < nt ? clamp_log_decay(to_f32(g[((int64_t)b * L + t0 + lane) * H + h])) : 0.0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const double end = __shfl_sync(0xffffffffu, sum, 31);
        cum[lane] = sum;
        eg[lane] = expf((float)sum);
        ek[lane] = expf((float)(end - sum));
        bt[lane] = lane < nt ? to_f32(beta[((int64_t)b * L + t0 + lane) * H + h]) : 0.f;
    }
    constexpr int kMine = kSeg / kWarps;  // tokens warp, warp + 8, ...: a batch of loads covers all of them
    for (int n = lane; n < NP; n += 32) {
        float kv[kMine], qv[kMine];
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            const int t = warp + kWarps * e;
            const int64_t at = (((int64_t)b * L + t0 + t) * G + grp) * N + n;
            kv[e] = t < nt && n < N ? to_f32(Bm[at]) : 0.f;
            qv[e] = t < nt && n < N ? to_f32(Cm[at]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kMine; ++e) ks[(warp + kWarps * e) * NP + n] = kv[e], qs[(warp + kWarps * e) * NP + n] = qv[e];
    }
    __syncthreads();
    {  // also z.err
        float d[kMine] = {};
#pragma unroll 2
        for (int p = lane; p < P; p += 32) {
            float ev[kMine], zv[kMine], yv[kMine];
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                const int t = warp + kWarps * e;
                const int64_t at = (((int64_t)b * L + t0 + t) * H + h) * P + p;
                ev[e] = t < nt ? err[at] : 0.f, zv[e] = t < nt ? zz[at] : 0.f, yv[e] = t < nt ? to_f32(dy[at]) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                const int t = warp + kWarps * e;
                dyT[p * kTp + t] = yv[e];
                uT[p * kTp + t] = bt[t] * ev[e];
                rT[p * kTp + t] = bt[t] * zv[e];
                if (kParts && t < nt) store_as(dx + (((int64_t)b * L + t0 + t) * H + h) * P + p, bt[t] * zv[e]);
                d[e] = fmaf(zv[e], ev[e], d[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            d[e] = warp_sum(d[e]);
            if (lane == 0) zd[warp + kWarps * e] = d[e];
        }
    }
    __syncthreads();
    if (tid < nt) store_as(dbeta + ((int64_t)b * L + t0 + tid) * H + h, zd[tid]);
    {  // pairs: tokens i = 4 warp .. + 3 by j = lane
        float dp[4] = {0.f, 0.f, 0.f, 0.f}, dm[4] = {0.f, 0.f, 0.f, 0.f}, qk[4] = {0.f, 0.f, 0.f, 0.f}, kk[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int p = 0; p < P; ++p) {
            const float4 y = *reinterpret_cast<const float4 *>(dyT + p * kTp + 4 * warp);
            const float4 r = *reinterpret_cast<const float4 *>(rT + p * kTp + 4 * warp);
            const float u = uT[p * kTp + lane];
            dp[0] = fmaf(y.x, u, dp[0]), dp[1] = fmaf(y.y, u, dp[1]), dp[2] = fmaf(y.z, u, dp[2]), dp[3] = fmaf(y.w, u, dp[3]);
            dm[0] = fmaf(r.x, u, dm[0]), dm[1] = fmaf(r.y, u, dm[1]), dm[2] = fmaf(r.z, u, dm[2]), dm[3] = fmaf(r.w, u, dm[3]);
        }
        for (int n = 0; n < N; n += 4) {  // (zeros past N)
            const float4 kj = *reinterpret_cast<const float4 *>(ks + lane * NP + n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 qi = *reinterpret_cast<const float4 *>(qs + (4 * warp + e) * NP + n);
                const float4 ki = *reinterpret_cast<const float4 *>(ks + (4 * warp + e) * NP + n);
                qk[e] = fmaf(qi.x, kj.x, fmaf(qi.y, kj.y, fmaf(qi.z, kj.z, fmaf(qi.w, kj.w, qk[e]))));
                kk[e] = fmaf(ki.x, kj.x, fmaf(ki.y, kj.y, fmaf(ki.z, kj.z, fmaf(ki.w, kj.w, kk[e]))));
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * warp + e, j = lane;
            const float ex = j <= i ? expf((float)(cum[i] - cum[j])) : 0.f;
            const float pv = j <= i ? dp[e] * ex : 0.f, mv = j < i ? -dm[e] * ex : 0.f;
            wPt[j * kTp + i] = wP[i * kTp + j] = pv;
            pair[i * 33 + j] = pv * qk[e] + mv * kk[e];
            if (j < i) wM[i * kTp + j] = wM[j * kTp + i] = mv;
            if (j == i) wM[i * kTp + i] = 0.f;
        }
    }
    const int64_t seg_at = (((int64_t)b * H + h) * ns + c) * P * N;
    const float *S = seg_states + seg_at, *D = seg_cot + seg_at;
    const bool has_s = !kParts || seg_states, has_d = !kParts || seg_cot;  // (else zeros)
    const int tg = warp % Z::groups, ps = warp / Z::groups, tk0 = TK * tg;  // this warp's tokens; its share of the rows
    float2 fq[TK / 2][NJ], fk[TK / 2][NJ], fu[TK / 2][NJ];
#pragma unroll
    for (int t = 0; t < TK / 2; ++t)
#pragma unroll
        for (int j = 0; j < NJ; ++j) fq[t][j] = fk[t][j] = fu[t][j] = make_float2(0.f, 0.f);
    float ds = 0.f;
    const int p_end = P * (ps + 1) / PS;
    struct Rows {
        float s[Z::U][NJ], d[Z::U][NJ];
    };
    const auto load = [&](Rows &to, int p0) {
#pragma unroll
        for (int i = 0; i < Z::U; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = lane + 32 * j;
                const bool in = n < N && p0 + i < p_end;
                const int64_t at = in ? (int64_t)(p0 + i) * N + n : 0;
                to.s[i][j] = in && has_s ? S[at] : 0.f;
                to.d[i][j] = in && has_d ? D[at] : 0.f;
            }
    };
    Rows next;
    load(next, P * ps / PS);
    for (int p0 = P * ps / PS; p0 < p_end; p0 += Z::U) {  // the next rows are on their way
        const Rows now = next;
        load(next, p0 + Z::U);
#pragma unroll
        for (int i = 0; i < Z::U; ++i) {
            const int p = p0 + i;
            if (p >= p_end) break;
#pragma unroll
            for (int t = 0; t < TK; t += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(dyT + p * kTp + tk0 + t);
                const float4 r = *reinterpret_cast<const float4 *>(rT + p * kTp + tk0 + t);
                const float4 u = *reinterpret_cast<const float4 *>(uT + p * kTp + tk0 + t);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float2 sv = both(now.s[i][j]), dv = both(now.d[i][j]);
                    fq[t / 2][j] = fma2(low2(y), sv, fq[t / 2][j]), fq[t / 2 + 1][j] = fma2(high2(y), sv, fq[t / 2 + 1][j]);
                    fk[t / 2][j] = fma2(low2(r), sv, fk[t / 2][j]), fk[t / 2 + 1][j] = fma2(high2(r), sv, fk[t / 2 + 1][j]);
                    fu[t / 2][j] = fma2(low2(u), dv, fu[t / 2][j]), fu[t / 2 + 1][j] = fma2(high2(u), dv, fu[t / 2 + 1][j]);
                }
            }
            if (tg == 0)
#pragma unroll
                for (int j = 0; j < NJ; ++j) ds = fmaf(now.s[i][j], now.d[i][j], ds);
        }
    }
    // dg's terms with S and D, as far as these rows go: per token, and the end's
    float tok[2][TK], end = eg[kSeg - 1] * ds;
#pragma unroll
    for (int t = 0; t < TK; t += 2) {
        float d[2] = {0.f, 0.f}, U[2] = {0.f, 0.f};
        const float e0 = eg[tk0 + t], e1 = eg[tk0 + t + 1], k0 = ek[tk0 + t], k1 = ek[tk0 + t + 1];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = lane + 32 * j;
            const bool in = n < N;
            const float2 q2 = make_float2(in ? qs[(tk0 + t) * NP + n] : 0.f, in ? qs[(tk0 + t + 1) * NP + n] : 0.f);
            const float2 n2 = make_float2(in ? ks[(tk0 + t) * NP + n] : 0.f, in ? ks[(tk0 + t + 1) * NP + n] : 0.f);
            float2 &q = fq[t / 2][j], &k = fk[t / 2][j], &u = fu[t / 2][j];
            q.x *= e0, q.y *= e1, k.x *= e0, k.y *= e1, u.x *= k0, u.y *= k1;
            U[0] = fmaf(u.x, n2.x, U[0]), U[1] = fmaf(u.y, n2.y, U[1]);
            d[0] += q.x * q2.x - k.x * n2.x;
            d[1] += q.y * q2.y - k.y * n2.y;
            k.x = u.x - k.x, k.y = u.y - k.y;
        }
        tok[0][t] = d[0], tok[0][t + 1] = d[1], tok[1][t] = U[0], tok[1][t + 1] = U[1];
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < TK; ++t) {
            tok[m][t] = warp_sum(tok[m][t]);
            if (lane == 0) dots[m][ps][tk0 + t] = tok[m][t];
        }
    end = warp_sum(end);
    if (lane == 0) ends[warp] = end;
    __syncthreads();  // the pairs' weights are there
    // dQ += dP K, dK += dP^T Q + (dM + dM^T) K: this warp's share of the tokens j
    for (int i = kSeg * ps / PS; i < kSeg * (ps + 1) / PS; ++i) {
        float kn[NJ], qn[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = lane + 32 * j;
            kn[j] = n < N ? ks[i * NP + n] : 0.f;
            qn[j] = n < N ? qs[i * NP + n] : 0.f;
        }
#pragma unroll
        for (int t = 0; t < TK; t += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(wPt + i * kTp + tk0 + t);
            const float4 w = *reinterpret_cast<const float4 *>(wP + i * kTp + tk0 + t);
            const float4 m = *reinterpret_cast<const float4 *>(wM + i * kTp + tk0 + t);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                fq[t / 2][j] = fma2(low2(a), both(kn[j]), fq[t / 2][j]), fq[t / 2 + 1][j] = fma2(high2(a), both(kn[j]), fq[t / 2 + 1][j]);
                fk[t / 2][j] = fma2(low2(w), both(qn[j]), fk[t / 2][j]), fk[t / 2 + 1][j] = fma2(high2(w), both(qn[j]), fk[t / 2 + 1][j]);
                fk[t / 2][j] = fma2(low2(m), both(kn[j]), fk[t / 2][j]), fk[t / 2 + 1][j] = fma2(high2(m), both(kn[j]), fk[t / 2 + 1][j]);
            }
        }
    }
    if (warp == 0) {
        // a row of pairs per lane becomes its sums of columns before i, i up to the row's own token
        float run = 0.f;
        for (int i = 0; i < kSeg; ++i) {
            const float v = pair[lane * 33 + i];
            pair[lane * 33 + i] = i <= lane ? run : 0.f;
            run += v;
        }
        float after = 0.f, before = 0.f, d = 0.f;
        for (int w = 0; w < PS; ++w) after += dots[0][w][lane], before += dots[1][w][lane];
        for (int w = 0; w < kWarps; ++w) d += ends[w];
        __syncwarp();
        for (int t = 0; t < kSeg; ++t) d += pair[t * 33 + lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {  // the tokens from this one to the end; those up to this one
            const float a = __shfl_down_sync(0xffffffffu, after, o), u = __shfl_up_sync(0xffffffffu, before, o);
            if (lane + o < 32) after += a;
            if (lane >= o) before += u;
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);  // (without this one)
        if (lane < nt) store_as(dg + ((int64_t)b * L + t0 + lane) * H + h, d + after + (lane ? before : 0.f));
    }
    if constexpr (PS > 1) {  // the other half's sums, through shared memory (all of which is free now)
        __syncthreads();
        float4 *buf = reinterpret_cast<float4 *>(sm) + tg * (TK / 2 * NJ * 32) + lane;
        if (ps == 1)
#pragma unroll
            for (int t = 0; t < TK / 2; ++t)
#pragma unroll
                for (int j = 0; j < NJ; ++j) buf[(t * NJ + j) * 32] = make_float4(fq[t][j].x, fq[t][j].y, fk[t][j].x, fk[t][j].y);
        __syncthreads();
        if (ps == 1) return;
#pragma unroll
        for (int t = 0; t < TK / 2; ++t)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float4 o = buf[(t * NJ + j) * 32];
                fq[t][j].x += o.x, fq[t][j].y += o.y, fk[t][j].x += o.z, fk[t][j].y += o.w;
            }
    }
#pragma unroll
    for (int t = 0; t < TK; ++t) {
        if (tk0 + t >= nt) continue;
        const int64_t at = (((int64_t)b * L + t0 + tk0 + t) * H + h) * N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = lane + 32 * j;
            if (n >= N) continue;
            dC_part[at + n] = t & 1 ? fq[t / 2][j].y : fq[t / 2][j].x;
            dB_part[at + n] = t & 1 ? fk[t / 2][j].y : fk[t / 2][j].x;
        }
    }
}

// Sums over the `per` heads of each group, in head order; a thread takes V columns of a row (token, group), whose
// heads' rows stand one after another.
template <typename T, int V>
__global__ void __launch_bounds__(kThr)
    k_delta_group_sum(const float *__restrict__ dB_part, const float *__restrict__ dC_part, int64_t rows, int per, int N,
                      T *__restrict__ dBm, T *__restrict__ dCm) {
    const int nv = N / V, at_once = kThr / nv, mine = threadIdx.x / nv, c = threadIdx.x % nv * V;
    if (mine >= at_once) return;
    for (int64_t row = (int64_t)blockIdx.x * at_once + mine; row < rows; row += (int64_t)gridDim.x * at_once) {
        float sb[V], sc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sb[e] = sc[e] = 0.f;
        for (int j = 0; j < per; ++j) {
            const int64_t at = (row * per + j) * N + c;
            float fb[V], fc[V];
            if constexpr (V == 4) {
                *reinterpret_cast<float4 *>(fb) = *reinterpret_cast<const float4 *>(dB_part + at);
                *reinterpret_cast<float4 *>(fc) = *reinterpret_cast<const float4 *>(dC_part + at);
            } else {
                fb[0] = dB_part[at], fc[0] = dC_part[at];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) sb[e] += fb[e], sc[e] += fc[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            store_as(dBm + row * N + c + e, sb[e]);
            store_as(dCm + row * N + c + e, sc[e]);
        }
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
    dim3 grid((unsigned)((p.P + kSeqRows - 1) / kSeqRows), (unsigned)p.H, (unsigned)p.B);
    const auto kernel = p.y ? k_delta_seq<T, NJ, true> : k_delta_seq<T, NJ, false>;
    kernel<<<grid, kSeqThr, 0, s>>>(static_cast<const T *>(p.x), static_cast<const T *>(p.g), static_cast<const T *>(p.beta),
                                    static_cast<const T *>(p.Bm), p.y ? static_cast<const T *>(p.Cm) : nullptr, p.h0, p.L,
                                    (int)p.H, (int)p.P, (int)p.G, (int)p.N, static_cast<T *>(p.y), p.h_final, seg_states, err);
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
    dim3 grid((unsigned)((p.P + kSeqRows - 1) / kSeqRows), (unsigned)p.H, (unsigned)p.B);
    k_delta_seq_bwd<T, NJ><<<grid, kSeqThr, 0, s>>>(static_cast<const T *>(gr.dy), gr.dh_final, static_cast<const T *>(p.g),
                                                 static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
                                                 static_cast<const T *>(p.Cm), p.L, (int)p.H, (int)p.P, (int)p.G, (int)p.N,
                                                 static_cast<T *>(gr.dx), z, seg_cot, gr.dh0);
    return cudaGetLastError();
}

template <int NJ>
size_t grads_smem(const DeltaProblem &p) {
    const size_t tiles = 3 * p.P * kTp + 2 * kSeg * grads_stride((int)p.N) + 3 * kSeg * kTp + kSeg * 33;
    const size_t joined = GradsTile<NJ>::split > 1 ? (size_t)kSeg * NJ * 32 * 2 : 0;  // dQ and dK of half of the warps
    return sizeof(float) * (tiles > joined ? tiles : joined);
}

template <typename T, int NJ, bool kParts>
cudaError_t grads_launch(const DeltaProblem &p, const DeltaGrads &gr, const float *states, const float *cot, Row<T, kParts> err,
                         Row<T, kParts> z, float *dB, float *dC, cudaStream_t s) {
    const size_t smem = grads_smem<NJ>(p);
    const cudaError_t e = cudaFuncSetAttribute(k_delta_grads<T, NJ, kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e) return e;
    dim3 grid((unsigned)((p.L + kSeg - 1) / kSeg), (unsigned)p.H, (unsigned)p.B);
    k_delta_grads<T, NJ, kParts><<<grid, kThr, smem, s>>>(
        static_cast<const T *>(gr.dy), static_cast<const T *>(p.g), static_cast<const T *>(p.beta), static_cast<const T *>(p.Bm),
        static_cast<const T *>(p.Cm), states, cot, err, z, p.L, (int)p.H, (int)p.P, (int)p.G, (int)p.N, dB, dC,
        static_cast<T *>(gr.dg), static_cast<T *>(gr.dbeta), static_cast<T *>(gr.dx));
    return cudaGetLastError();
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
    const auto both_of = [&](auto nj) {
        constexpr int NJ = decltype(nj)::value;
        const cudaError_t f = seq_bwd_launch<T, NJ>(p, gr, z, cot, s);
        return f ? f : grads_launch<T, NJ, false>(p, gr, states, cot, Row<T, false>{err}, Row<T, false>{z}, dB, dC, s);
    };
    if (p.N <= 32) e = both_of(std::integral_constant<int, 1>());
    else if (p.N <= 64) e = both_of(std::integral_constant<int, 2>());
    else if (p.N <= 128) e = both_of(std::integral_constant<int, 4>());
    else e = both_of(std::integral_constant<int, 8>());
    if (e) return e;
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
    const int64_t rows = p.B * p.L * p.G;
    const int V = p.N % 4 ? 1 : 4, at_once = (int)(kThr / (p.N / V));
    const int64_t blocks = (rows + at_once - 1) / at_once;
    const int64_t most = (int64_t)sm_count() * 8;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    const auto go = [&](auto kernel, auto *b, auto *c) {
        kernel<<<grid, kThr, 0, s>>>(dB_part, dC_part, rows, (int)(p.H / p.G), (int)p.N, b, c);
    };
    using bf = __nv_bfloat16;
    if (p.dtype == SSD_F32)
        go(V == 4 ? k_delta_group_sum<float, 4> : k_delta_group_sum<float, 1>, static_cast<float *>(dBm), static_cast<float *>(dCm));
    else
        go(V == 4 ? k_delta_group_sum<bf, 4> : k_delta_group_sum<bf, 1>, static_cast<bf *>(dBm), static_cast<bf *>(dCm));
    return cudaGetLastError();
}

cudaError_t delta_seq_fwd(const DeltaProblem &p, cudaStream_t s) {
    return p.dtype == SSD_F32 ? seq_typed<float>(p, nullptr, nullptr, s) : seq_typed<__nv_bfloat16>(p, nullptr, nullptr, s);
}

cudaError_t delta_short_grads(const DeltaProblem &p, const DeltaGrads &g, const DeltaParts &parts, float *dB, float *dC,
                              cudaStream_t s) {
    using bf = __nv_bfloat16;
    const Row<bf, true> err{static_cast<const bf *>(parts.err), static_cast<const bf *>(parts.err_lo)};
    const Row<bf, true> z{static_cast<const bf *>(parts.z), static_cast<const bf *>(parts.z_lo)};
    if (p.N <= 32) return grads_launch<bf, 1, true>(p, g, p.h0, g.dh_final, err, z, dB, dC, s);
    if (p.N <= 64) return grads_launch<bf, 2, true>(p, g, p.h0, g.dh_final, err, z, dB, dC, s);
    return grads_launch<bf, 4, true>(p, g, p.h0, g.dh_final, err, z, dB, dC, s);
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
