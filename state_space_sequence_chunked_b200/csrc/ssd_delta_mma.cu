// The gated delta rule on tensor cores, chunked: bf16 inputs, dstate <= 128 and headdim in multiples
// of 8. With cum the cumulated log decay in a chunk of 64 tokens, E_ij = exp(cum_i - cum_j),
// M = tril(K K^T o E, -1), and W the strictly lower solution of W = -M (I + diag(beta) W):
//     R = X - exp(cum) K S^T,   err = R + W (beta R),   u = beta err,
//     Y = exp(cum) Q S^T + tril(Q K^T o E) u,   S <- exp(cum_end) S + u^T (exp(cum_end - cum) K)
// (K, Q: keys Bm and queries Cm; the inverse (I + M diag(beta))^-1 is I + W diag(beta), so no division by
// beta is needed and its unit diagonal is exact).
//
//   k_delta_prep   everything that does not depend on the state: W and tril(Q K^T o E) per chunk and
//                  head, all chunks at once, as the register fragments the chain multiplies by.
//   k_delta_chain  the chain over the chunks. The rows p of the state are independent given K, Q
//                  and W, so a warp keeps 16 rows of it in fp32 accumulators for the whole sequence
//                  and nothing crosses warps: the accumulators of one product are, in place, the left
//                  operand of the next (mma.sync m16n8k16: both layouts hold the same elements), and
//                  tokens are the columns throughout (R^T, u^T, Y^T).
//
// Precision. The final state is fp32, so what enters it is kept to 2^-16: an fp32 left operand is
// split in two bf16 parts (hi + lo) and W too (three products); K, Q are exact. Y is rounded to bf16,
// so S and tril(Q K^T o E) enter it as one bf16 part, u as two.
//
// mma.sync because the chain is one of dependent small products: with the state in registers a chunk
// costs no shared-memory or tensor-memory round trip between them. m16n8k16 measures 550 TFLOP/s
// on this part (8.4 cycles per instruction and sub-partition).
#include "ssd_delta.cuh"

namespace ssd {
namespace {

constexpr int kC = kDeltaChunk;  // tokens per chunk
constexpr int kThr = 128;        // 4 warps
constexpr int kRowsCta = 64;     // state rows per CTA of the chain

// Blocks (a, b) of 16 x 16 tokens with a >= b, in the order a (a + 1) / 2 + b.
constexpr int kBlocks = 10;
__host__ __device__ constexpr int block_at(int a, int b) { return a * (a + 1) / 2 + b; }

// Per chunk and head, in the workspace: fragments as right operands, one 16-byte vector per lane and
// block, and the scalars exp(cum), exp(cum_end - cum), beta of the chunk's tokens, then cum as a sum of
// two floats. The forward has W (hi, lo), the scalars and the masked Q K^T; the backward pass W, the
// scalars, and both transposed (hi, lo).
constexpr int kFragBytes = 512;  // one vector per lane
constexpr int kWBytes = kBlocks * 2 * kFragBytes;
constexpr int kPBytes = kBlocks * kFragBytes;
constexpr int kScalBytes = 5 * kC * 4;
template <bool BWD>
struct Prep {
    static constexpr int W = 0, scal = kWBytes, P = scal + kScalBytes, WT = scal + kScalBytes, PT = WT + kWBytes;
    static constexpr int bytes = BWD ? PT + kWBytes : P + kPBytes;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r0), "r"(r1), "r"(r2),
                 "r"(r3)
                 : "memory");
}
__device__ __forceinline__ uint32_t trans8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// hi + lo parts of a pair: what hi leaves of each value, rounded again (2^-17 of the value at worst).
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack(x, y);
    lo = pack(x - low(hi), y - high(hi));
}

// Left operand (16 x 16) from two neighbouring accumulator tiles: the same elements, converted.
__device__ __forceinline__ void split_a(const float (&t0)[4], const float (&t1)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split(t0[0], t0[1], hi[0], lo[0]);
    split(t0[2], t0[3], hi[1], lo[1]);
    split(t1[0], t1[1], hi[2], lo[2]);
    split(t1[2], t1[3], hi[3], lo[3]);
}

// Byte offset of 16-byte vector c of row r in a tile with rows of ROW bytes (a multiple of 128),
// swizzled so that the 8 rows of an 8 x 8 matrix fall in different banks.
template <int ROW>
__device__ __forceinline__ uint32_t at16(int r, int c) {
    return (uint32_t)(r * ROW + (((c & ~7) | ((c ^ r) & 7)) << 4));
}

// Loads kC tokens of [B, L, X, D] bf16 rows (head or group j, columns from d0) as a tile of NV vectors per row,
// zeros past the sequence and past D. D % 8 == 0.
template <int NV>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16 *__restrict__ src, int64_t b, int64_t L, int64_t t0,
                                          int X, int j, int D, int d0) {
    for (int i = threadIdx.x; i < kC * NV; i += kThr) {
        const int t = i / NV, c = i % NV;
        const bool in = t0 + t < L && d0 + 8 * c < D;
        const __nv_bfloat16 *p = in ? src + ((b * L + t0 + t) * X + j) * (int64_t)D + d0 + 8 * c : src;
        cp16(dst + at16<NV * 16>(t, c), p, in);
    }
}

// ---------------------------------------------------------------------------------------------
// k_delta_prep: grid (chunks, G * slices, B); a CTA forms K K^T and Q K^T of one chunk and group once (a warp
// per 16 rows), then a warp takes a head at a time. Per head: the diagonal blocks of W by substitution
// in fp32 (a lane per column), then the rows of blocks below, on tensor cores with every fp32 operand
// in two bf16 parts:
//     W_ab = -(I + W_aa diag(beta_a)) (M_ab (I + diag(beta_b) W_bb) + sum_{b<c<a} M_ac diag(beta_c) W_cb).
constexpr int kLd = kC + 4;  // padded row of the fp32 tiles
constexpr int kDl = 20;      // padded row of a diagonal block

struct PrepWarp {
    float diag[4][16 * kDl];
    float2 cum[kC];  // cum as a sum of two floats
    float beta[kC];
};
template <int NT>
struct PrepSmem {
    float kk[kC * kLd], qk[kC * kLd];
    union {
        struct {
            __nv_bfloat16 k[kC * NT], q[kC * NT];
        };
        PrepWarp w[4];
    };
};

__device__ __forceinline__ float decay_between(float2 i, float2 j) { return __expf((i.x - j.x) + (i.y - j.y)); }

// Right-operand fragments (hi, lo) of a 16 x 16 fp32 block in accumulator layout, rows g and g + 8 scaled.
__device__ __forceinline__ void split_b(const float (&b)[2][4], float s0, float s1, uint32_t (&h)[4], uint32_t (&l)[4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        split(s0 * b[n][0], s0 * b[n][1], h[2 * n], l[2 * n]);
        split(s1 * b[n][2], s1 * b[n][3], h[2 * n + 1], l[2 * n + 1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = trans8(h[e]), l[e] = trans8(l[e]);
}
__device__ __forceinline__ void block_mma(float (&acc)[2][4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma(acc[n], al, bh[2 * n], bh[2 * n + 1]);
        mma(acc[n], ah, bl[2 * n], bl[2 * n + 1]);
        mma(acc[n], ah, bh[2 * n], bh[2 * n + 1]);
    }
}

// Fragments of block `at` of W, and for the backward pass of its transpose.
template <bool BWD>
__device__ __forceinline__ void put_w(char *out, int at, int lane, const float (&w)[2][4]) {
    uint32_t hi[4], lo[4];  // rows 0-7: two halves of the columns, then rows 8-15
    split(w[0][0], w[0][1], hi[0], lo[0]);
    split(w[1][0], w[1][1], hi[1], lo[1]);
    split(w[0][2], w[0][3], hi[2], lo[2]);
    split(w[1][2], w[1][3], hi[3], lo[3]);
    uint4 *o = reinterpret_cast<uint4 *>(out + Prep<BWD>::W) + at * 64 + lane;
    o[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    o[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if constexpr (BWD) {
        o = reinterpret_cast<uint4 *>(out + Prep<BWD>::WT) + at * 64 + lane;
        o[0] = make_uint4(trans8(hi[0]), trans8(hi[2]), trans8(hi[1]), trans8(hi[3]));
        o[32] = make_uint4(trans8(lo[0]), trans8(lo[2]), trans8(lo[1]), trans8(lo[3]));
    }
}

template <int NT, bool BWD>
__global__ void __launch_bounds__(kThr)
    k_delta_prep(const __nv_bfloat16 *__restrict__ Bm, const __nv_bfloat16 *__restrict__ Cm, const __nv_bfloat16 *__restrict__ g,
                 const __nv_bfloat16 *__restrict__ beta, int64_t L, int H, int G, int N, int slices, char *__restrict__ ws) {
    extern __shared__ __align__(128) char raw[];
    PrepSmem<NT> &sm = *reinterpret_cast<PrepSmem<NT> *>(raw);
    using Lay = Prep<BWD>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tg = lane & 3;
    const int64_t c = blockIdx.x, nc = gridDim.x, b = blockIdx.z, t0 = c * kC;
    const int grp = blockIdx.y / slices, slice = blockIdx.y % slices, per = H / G;
    const int h_begin = grp * per + per * slice / slices, h_end = grp * per + per * (slice + 1) / slices;
    const uint32_t ka = smem_addr(sm.k), qa = smem_addr(sm.q);
    load_tile<NT / 8>(ka, Bm, b, L, t0, G, grp, N, 0);
    load_tile<NT / 8>(qa, Cm, b, L, t0, G, grp, N, 0);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    {  // rows 16 warp .. + 15 of K K^T and Q K^T, columns up to the diagonal block
        float kk[8][4], qk[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
#pragma unroll
        for (int s = 0; s < NT / 16; ++s) {
            uint32_t ak[4], aq[4];
            const int row = 16 * warp + (lane & 15), ch = 2 * s + (lane >> 4);
            ldsm4(ak, ka + at16<NT * 2>(row, ch));
            ldsm4(aq, qa + at16<NT * 2>(row, ch));
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (jj <= warp) {
                    uint32_t bk[4];
                    ldsm4(bk, ka + at16<NT * 2>(16 * jj + (lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
                    mma(kk[2 * jj], ak, bk[0], bk[1]);
                    mma(kk[2 * jj + 1], ak, bk[2], bk[3]);
                    mma(qk[2 * jj], aq, bk[0], bk[1]);
                    mma(qk[2 * jj + 1], aq, bk[2], bk[3]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < 2 * warp + 2) {
                const int i = 16 * warp + gr, col = 8 * j + 2 * tg;
                *reinterpret_cast<float2 *>(&sm.kk[i * kLd + col]) = make_float2(kk[j][0], kk[j][1]);
                *reinterpret_cast<float2 *>(&sm.kk[(i + 8) * kLd + col]) = make_float2(kk[j][2], kk[j][3]);
                *reinterpret_cast<float2 *>(&sm.qk[i * kLd + col]) = make_float2(qk[j][0], qk[j][1]);
                *reinterpret_cast<float2 *>(&sm.qk[(i + 8) * kLd + col]) = make_float2(qk[j][2], qk[j][3]);
            }
        }
    }
    __syncthreads();  // K and Q are done with: the warps' own memory lies over them
    PrepWarp &wm = sm.w[warp];
    for (int h = h_begin + warp; h < h_end; h += 4) {
        char *out = ws + ((b * H + h) * nc + c) * (int64_t)Lay::bytes;
        {  // cumulated log decay: 2 tokens per lane, fp64
            const int64_t at = (b * L + t0 + 2 * lane) * H + h;
            const bool in0 = t0 + 2 * lane < L, in1 = t0 + 2 * lane + 1 < L;
            const double g0 = in0 ? clamp_log_decay(to_f32(g[at])) : 0.0, g1 = in1 ? clamp_log_decay(to_f32(g[at + H])) : 0.0;
            const float b0 = in0 ? to_f32(beta[at]) : 0.f, b1 = in1 ? to_f32(beta[at + H]) : 0.f;
            double sum = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double total = __shfl_sync(0xffffffffu, sum, 31), first = sum - g1;
            const float f0 = (float)first, f1 = (float)sum, l0 = (float)(first - (double)f0), l1 = (float)(sum - (double)f1);
            wm.cum[2 * lane] = make_float2(f0, l0);
            wm.cum[2 * lane + 1] = make_float2(f1, l1);
            wm.beta[2 * lane] = b0, wm.beta[2 * lane + 1] = b1;
            float2 *scal = reinterpret_cast<float2 *>(out + Lay::scal) + lane;
            scal[0] = make_float2(expf(f0), expf(f1));
            scal[kC / 2] = make_float2(expf((float)(total - first)), expf((float)(total - sum)));
            scal[kC] = make_float2(b0, b1);
            scal[3 * kC / 2] = make_float2(f0, f1);
            scal[2 * kC] = make_float2(l0, l1);
        }
        __syncwarp();
        // block (a, cc): M in accumulator layout; the masked Q K^T goes out
        const auto block = [&](int a, int cc, float (&m)[2][4]) {
            float p[2][4];
            const float2 ri[2] = {wm.cum[16 * a + gr], wm.cum[16 * a + gr + 8]};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int j = 16 * cc + 8 * n + 2 * tg;
                const float4 cj = *reinterpret_cast<const float4 *>(&wm.cum[j]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = 16 * a + gr + 8 * r;
                    const float2 kk = *reinterpret_cast<const float2 *>(&sm.kk[i * kLd + j]);
                    const float2 qk = *reinterpret_cast<const float2 *>(&sm.qk[i * kLd + j]);
                    const float e0 = j <= i ? decay_between(ri[r], make_float2(cj.x, cj.y)) : 0.f;
                    const float e1 = j + 1 <= i ? decay_between(ri[r], make_float2(cj.z, cj.w)) : 0.f;
                    m[n][2 * r] = j < i ? kk.x * e0 : 0.f, m[n][2 * r + 1] = j + 1 < i ? kk.y * e1 : 0.f;
                    p[n][2 * r] = j <= i ? qk.x * e0 : 0.f, p[n][2 * r + 1] = j + 1 <= i ? qk.y * e1 : 0.f;
                }
            }
            if constexpr (BWD) {
                uint32_t ph[4], pl[4];
                split_b(p, 1.f, 1.f, ph, pl);
                uint4 *o = reinterpret_cast<uint4 *>(out + Lay::PT) + block_at(a, cc) * 64 + lane;
                o[0] = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                o[32] = make_uint4(pl[0], pl[1], pl[2], pl[3]);
            } else {
                reinterpret_cast<uint4 *>(out + Lay::P)[block_at(a, cc) * 32 + lane] =
                    make_uint4(pack(p[0][0], p[0][1]), pack(p[1][0], p[1][1]), pack(p[0][2], p[0][3]), pack(p[1][2], p[1][3]));
            }
        };
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float m[2][4];
            block(a, a, m);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<float2 *>(&wm.diag[a][(gr + 8 * r) * kDl + 8 * n + 2 * tg]) =
                        make_float2(m[n][2 * r], m[n][2 * r + 1]);
        }
        __syncwarp();
        // a half warp per diagonal block, a lane per column: w_i = -m_ij - sum_{j<k<i} m_ik beta_k w_k
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int a = 2 * half + (lane >> 4), j = lane & 15;
            float *m = wm.diag[a];
            float w[16], bw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float row[16];
#pragma unroll
                for (int k = 0; k < (i + 3) / 4; ++k) *reinterpret_cast<float4 *>(row + 4 * k) = *reinterpret_cast<const float4 *>(m + i * kDl + 4 * k);
                float s0 = m[i * kDl + j], s1 = 0.f;
#pragma unroll
                for (int k = 0; k < i; ++k) (k & 1 ? s1 : s0) = fmaf(row[k], bw[k], k & 1 ? s1 : s0);
                w[i] = i > j ? -(s0 + s1) : 0.f;
                bw[i] = wm.beta[16 * a + i] * w[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) m[i * kDl + j] = w[i];
        }
        __syncwarp();
        uint32_t bh[6][4], bl[6][4];  // diag(beta) W_cb, c <= 2, as right operands
        const auto diag = [&](int a, float (&d)[2][4]) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 v = *reinterpret_cast<const float2 *>(&wm.diag[a][(gr + 8 * r) * kDl + 8 * n + 2 * tg]);
                    d[n][2 * r] = v.x, d[n][2 * r + 1] = v.y;
                }
        };
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float m[3][2][4], d[2][4];
            uint32_t mh[3][4], ml[3][4], dh[4], dl[4];
            diag(a, d);
            put_w<BWD>(out, block_at(a, a), lane, d);
            const float s0 = wm.beta[16 * a + gr], s1 = wm.beta[16 * a + gr + 8];
            if (a < 3) split_b(d, s0, s1, bh[block_at(a, a)], bl[block_at(a, a)]);
            if (a == 0) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 bj = *reinterpret_cast<const float2 *>(&wm.beta[16 * a + 8 * n + 2 * tg]);
                d[n][0] *= bj.x, d[n][1] *= bj.y, d[n][2] *= bj.x, d[n][3] *= bj.y;
            }
            split_a(d[0], d[1], dh, dl);
#pragma unroll
            for (int cc = 0; cc < a; ++cc) {
                block(a, cc, m[cc]);
                split_a(m[cc][0], m[cc][1], mh[cc], ml[cc]);
            }
#pragma unroll
            for (int bb = 0; bb < a; ++bb) {
                float u[2][4], w[2][4];
                uint32_t uh[4], ul[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[n][e] = m[bb][n][e];
#pragma unroll
                for (int cc = bb; cc < a; ++cc) block_mma(u, mh[cc], ml[cc], bh[block_at(cc, bb)], bl[block_at(cc, bb)]);
                split_b(u, 1.f, 1.f, uh, ul);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[n][e] = u[n][e];
                block_mma(w, dh, dl, uh, ul);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[n][e] = -w[n][e];
                put_w<BWD>(out, block_at(a, bb), lane, w);
                if (a < 3) split_b(w, s0, s1, bh[block_at(a, bb)], bl[block_at(a, bb)]);
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------------------------
// k_delta_chain: grid (ceil(P / 64), H, B), a warp per 16 state rows, two stages of a chunk's operands
// loaded ahead with cp.async.
template <int NT>
struct ChainStage {
    __nv_bfloat16 k[kC * NT], q[kC * NT], x[kC * kRowsCta];
    char prep[Prep<false>::bytes];
};

template <int NT>
__global__ void __launch_bounds__(kThr, 2)
    k_delta_chain(const __nv_bfloat16 *__restrict__ x, const __nv_bfloat16 *__restrict__ Bm, const __nv_bfloat16 *__restrict__ Cm,
                  const float *__restrict__ h0, const char *__restrict__ ws, int64_t L, int H, int P, int G, int N,
                  __nv_bfloat16 *__restrict__ y, float *__restrict__ h_final) {
    extern __shared__ __align__(128) char raw[];
    ChainStage<NT> *stages = reinterpret_cast<ChainStage<NT> *>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tg = lane & 3;
    const int h = blockIdx.y, grp = h / (H / G), pc = blockIdx.x * kRowsCta, p0 = pc + 16 * warp;
    const int64_t b = blockIdx.z, nc = (L + kC - 1) / kC;
    const bool on = p0 < P;  // a warp with rows
    constexpr int kPrepBytes = Prep<false>::bytes;
    const char *prep = ws + (b * H + h) * nc * (int64_t)kPrepBytes;

    const auto load = [&](int64_t c) {
        ChainStage<NT> &st = stages[c & 1];
        load_tile<NT / 8>(smem_addr(st.k), Bm, b, L, c * kC, G, grp, N, 0);
        load_tile<NT / 8>(smem_addr(st.q), Cm, b, L, c * kC, G, grp, N, 0);
        load_tile<kRowsCta / 8>(smem_addr(st.x), x, b, L, c * kC, H, h, P, pc);
        const uint32_t dst = smem_addr(st.prep);
        for (int i = tid; i < kPrepBytes / 16; i += kThr) cp16(dst + 16 * i, prep + c * kPrepBytes + 16 * i, true);
        cp_commit();
    };
    load(0);

    // state rows p0 + gr and p0 + gr + 8, columns 8 j + 2 tg and + 1
    float S[NT / 8][4];
    const int64_t row = (b * H + h) * (int64_t)P + p0 + gr;
#pragma unroll
    for (int j = 0; j < NT / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = 8 * j + 2 * tg + (e & 1), r = 8 * (e >> 1);
            S[j][e] = h0 && n < N && p0 + gr + r < P ? h0[(row + r) * N + n] : 0.f;
        }

    for (int64_t c = 0; c < nc; ++c) {
        if (c + 1 < nc) {
            load(c + 1);
            cp_wait<1>();
        } else {
            cp_wait<0>();
        }
        __syncthreads();
        ChainStage<NT> &st = stages[c & 1];
        if (on) {
            const uint32_t ka = smem_addr(st.k), qa = smem_addr(st.q), xa = smem_addr(st.x);
            const uint4 *wf = reinterpret_cast<const uint4 *>(st.prep) + lane;
            const uint4 *pf = reinterpret_cast<const uint4 *>(st.prep + Prep<false>::P) + lane;
            const float *eg = reinterpret_cast<const float *>(st.prep + Prep<false>::scal), *ek = eg + kC, *bt = eg + 2 * kC;
            float R[8][4], Y[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) R[j][e] = Y[j][e] = 0.f;
            // S K^T and S Q^T
#pragma unroll
            for (int s = 0; s < NT / 16; ++s) {
                uint32_t hi[4], lo[4];
                split_a(S[2 * s], S[2 * s + 1], hi, lo);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    uint32_t bk[4], bq[4];
                    const uint32_t off = at16<NT * 2>(16 * jj + (lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1));
                    ldsm4(bk, ka + off);
                    ldsm4(bq, qa + off);
                    mma(R[2 * jj], lo, bk[0], bk[1]);
                    mma(R[2 * jj + 1], lo, bk[2], bk[3]);
                    mma(Y[2 * jj], hi, bq[0], bq[1]);
                    mma(Y[2 * jj + 1], hi, bq[2], bq[3]);
                    mma(R[2 * jj], hi, bk[0], bk[1]);
                    mma(R[2 * jj + 1], hi, bk[2], bk[3]);
                }
            }
            // R = X - exp(cum) S K^T, and exp(cum) S Q^T
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t xf[4];
                ldsm4t(xf, xa + at16<kRowsCta * 2>(16 * jj + (lane & 7) + ((lane >> 4) << 3), 2 * warp + ((lane >> 3) & 1)));
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = 2 * jj + n;
                    const float2 e = *reinterpret_cast<const float2 *>(eg + 8 * j + 2 * tg);
                    R[j][0] = fmaf(-e.x, R[j][0], low(xf[2 * n]));
                    R[j][1] = fmaf(-e.y, R[j][1], high(xf[2 * n]));
                    R[j][2] = fmaf(-e.x, R[j][2], low(xf[2 * n + 1]));
                    R[j][3] = fmaf(-e.y, R[j][3], high(xf[2 * n + 1]));
                    Y[j][0] *= e.x, Y[j][1] *= e.y, Y[j][2] *= e.x, Y[j][3] *= e.y;
                }
            }
            // err = R + W (beta R): the blocks of a column of tokens at a time, from the last column on, so
            // that R can take the sums in place (block row a needs the beta R of blocks b <= a only)
            uint32_t ah[4][4], al[4][4];
#pragma unroll
            for (int bb = 0; bb < 4; ++bb) {
                float t[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 e = *reinterpret_cast<const float2 *>(bt + 16 * bb + 8 * n + 2 * tg);
                    t[n][0] = e.x * R[2 * bb + n][0], t[n][1] = e.y * R[2 * bb + n][1];
                    t[n][2] = e.x * R[2 * bb + n][2], t[n][3] = e.y * R[2 * bb + n][3];
                }
                split_a(t[0], t[1], ah[bb], al[bb]);
            }
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int bb = 0; bb <= a; ++bb) {
                    const uint4 wh = wf[block_at(a, bb) * 64], wl = wf[block_at(a, bb) * 64 + 32];
                    mma(R[2 * a], al[bb], wh.x, wh.y);
                    mma(R[2 * a + 1], al[bb], wh.z, wh.w);
                    mma(R[2 * a], ah[bb], wl.x, wl.y);
                    mma(R[2 * a + 1], ah[bb], wl.z, wl.w);
                    mma(R[2 * a], ah[bb], wh.x, wh.y);
                    mma(R[2 * a + 1], ah[bb], wh.z, wh.w);
                }
            // u = beta err; Y += tril(Q K^T o E) u
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 e = *reinterpret_cast<const float2 *>(bt + 8 * j + 2 * tg);
                R[j][0] *= e.x, R[j][1] *= e.y, R[j][2] *= e.x, R[j][3] *= e.y;
            }
#pragma unroll
            for (int bb = 0; bb < 4; ++bb) {
                uint32_t hi[4], lo[4];
                split_a(R[2 * bb], R[2 * bb + 1], hi, lo);
#pragma unroll
                for (int a = bb; a < 4; ++a) {
                    const uint4 f = pf[block_at(a, bb) * 32];
                    mma(Y[2 * a], lo, f.x, f.y);
                    mma(Y[2 * a + 1], lo, f.z, f.w);
                    mma(Y[2 * a], hi, f.x, f.y);
                    mma(Y[2 * a + 1], hi, f.z, f.w);
                }
            }
            // Y over this warp's columns of the x tile, then to memory
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
                stsm4t(xa + at16<kRowsCta * 2>(16 * jj + (lane & 7) + ((lane >> 4) << 3), 2 * warp + ((lane >> 3) & 1)),
                       pack(Y[2 * jj][0], Y[2 * jj][1]), pack(Y[2 * jj][2], Y[2 * jj][3]), pack(Y[2 * jj + 1][0], Y[2 * jj + 1][1]),
                       pack(Y[2 * jj + 1][2], Y[2 * jj + 1][3]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * i + (lane >> 1), v = 2 * warp + (lane & 1);
                const int64_t tt = c * kC + t;
                if (tt < L && pc + 8 * v < P)
                    *reinterpret_cast<uint4 *>(y + ((b * L + tt) * H + h) * (int64_t)P + pc + 8 * v) =
                        *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(st.x) + at16<kRowsCta * 2>(t, v));
            }
            // S <- exp(cum_end) S + (exp(cum_end - cum) u)^T K
            const float gamma = eg[kC - 1];
#pragma unroll
            for (int j = 0; j < NT / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[j][e] *= gamma;
#pragma unroll
            for (int bb = 0; bb < 4; ++bb) {
                uint32_t hi[4], lo[4];
                float t[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 e = *reinterpret_cast<const float2 *>(ek + 16 * bb + 8 * n + 2 * tg);
                    t[n][0] = e.x * R[2 * bb + n][0], t[n][1] = e.y * R[2 * bb + n][1];
                    t[n][2] = e.x * R[2 * bb + n][2], t[n][3] = e.y * R[2 * bb + n][3];
                }
                split_a(t[0], t[1], hi, lo);
#pragma unroll
                for (int j = 0; j < NT / 16; ++j) {
                    uint32_t bk[4];
                    ldsm4t(bk, ka + at16<NT * 2>(16 * bb + (lane & 15), 2 * j + (lane >> 4)));
                    mma(S[2 * j], lo, bk[0], bk[1]);
                    mma(S[2 * j + 1], lo, bk[2], bk[3]);
                    mma(S[2 * j], hi, bk[0], bk[1]);
                    mma(S[2 * j + 1], hi, bk[2], bk[3]);
                }
            }
        }
        __syncthreads();  // the stage is free
    }
    if (h_final && on) {
#pragma unroll
        for (int j = 0; j < NT / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = 8 * j + 2 * tg + (e & 1), r = 8 * (e >> 1);
                if (n < N && p0 + gr + r < P) h_final[(row + r) * N + n] = S[j][e];
            }
    }
}

template <int NT, bool BWD>
cudaError_t prep_launch(const DeltaProblem &p, char *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const int64_t nc = (p.L + kC - 1) / kC, units = nc * p.G * p.B;
    const int per = (int)(p.H / p.G);
    // a CTA walks all heads of a group while that leaves 3 CTAs (what fits) for every SM, and
    // four heads at least, one per warp
    int slices = units >= 148 * 3 ? 1 : (int)((148 * 3 + units - 1) / units);
    if (slices > (per + 3) / 4) slices = (per + 3) / 4;
    cudaError_t e;
    constexpr int smem = sizeof(PrepSmem<NT>);
    if ((e = cudaFuncSetAttribute(k_delta_prep<NT, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
    dim3 grid((unsigned)nc, (unsigned)(p.G * slices), (unsigned)p.B);
    k_delta_prep<NT, BWD><<<grid, kThr, smem, s>>>(static_cast<const bf *>(p.Bm), static_cast<const bf *>(p.Cm),
                                                   static_cast<const bf *>(p.g), static_cast<const bf *>(p.beta), p.L,
                                                   (int)p.H, (int)p.G, (int)p.N, slices, ws);
    return cudaGetLastError();
}

template <int NT>
cudaError_t fwd_launch(const DeltaProblem &p, char *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    cudaError_t e = prep_launch<NT, false>(p, ws, s);
    if (e) return e;
    constexpr int smem = 2 * sizeof(ChainStage<NT>);
    if ((e = cudaFuncSetAttribute(k_delta_chain<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
    dim3 grid((unsigned)((p.P + kRowsCta - 1) / kRowsCta), (unsigned)p.H, (unsigned)p.B);
    k_delta_chain<NT><<<grid, kThr, smem, s>>>(static_cast<const bf *>(p.x), static_cast<const bf *>(p.Bm),
                                               static_cast<const bf *>(p.Cm), p.h0, ws, p.L, (int)p.H, (int)p.P, (int)p.G,
                                               (int)p.N, static_cast<bf *>(p.y), p.h_final);
    return cudaGetLastError();
}

}  // namespace

bool delta_mma_supported(const DeltaProblem &p) {
    return p.dtype == SSD_BF16 && p.N <= 128 && p.N % 8 == 0 && p.P % 8 == 0 && p.L >= 8;
}

size_t delta_mma_fwd_workspace_bytes(const DeltaProblem &p) {
    return (size_t)(p.B * p.H) * (size_t)((p.L + kC - 1) / kC) * Prep<false>::bytes;
}

cudaError_t delta_mma_fwd(const DeltaProblem &p, void *ws, cudaStream_t s) {
    return p.N <= 64 ? fwd_launch<64>(p, static_cast<char *>(ws), s) : fwd_launch<128>(p, static_cast<char *>(ws), s);
}

}  // namespace ssd
