// The gated delta rule on tensor cores, chunked: bf16 inputs, dstate <= 128 (sizes that are no multiples of 8 on
// padded copies, at the end). With cum the cumulated log decay in a chunk of 64 tokens, E_ij = exp(cum_i - cum_j),
// M = tril(K K^T o E, -1), and W the strictly lower solution of W = -M (I + diag(beta) W):
//     R = X - exp(cum) K S^T,   err = R + W (beta R),   u = beta err,
//     Y = exp(cum) Q S^T + tril(Q K^T o E) u,   S <- exp(cum_end) S + u^T (exp(cum_end - cum) K)
// (K, Q: keys Bm and queries Cm; the inverse (I + M diag(beta))^-1 is I + W diag(beta), so no division by
// beta is needed and its unit diagonal is exact).
//
//   k_delta_prep (here)             what does not depend on the state: W, tril(Q K^T o E) and the decays per
//                                   chunk and head, all chunks at once, as right operands of the chain.
//   k_delta_tc    (ssd_delta_tc.cu) the chain over the chunks, the state in tensor memory.
//   k_delta_tc_bwd, k_delta_grads_tc  the backward pass: the states again and the chain in reverse, then what sums
//                                   over the rows of the state (ssd_delta_tc.cu, ssd_delta_grads.cu).
//
// Precision. The final state is fp32, so what enters it is kept to 2^-16: an fp32 left operand is
// split in two bf16 parts (hi + lo) and W too (three products); K, Q are exact. Y is rounded to bf16,
// so S and tril(Q K^T o E) enter it as one bf16 part, u as two: off by 2.4e-3 of its norm, where rounding it takes
// 1.7e-3. Two parts of each leave only that; they were timed at 145 us against 141 (24 heads, 8 x 2048 tokens)
// and, with 168 MB more of workspace written and read, at 682 against 615 (80 heads, 4 x 8192).
#include "delta_tc.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kThr = 128;  // 4 warps

// Blocks (a, b) of 16 x 16 tokens with a >= b, in the order a (a + 1) / 2 + b.
constexpr int kBlocks = 10;
__host__ __device__ constexpr int block_at(int a, int b) { return a * (a + 1) / 2 + b; }

// Per chunk and head, in the workspace. First what k_delta_tc loads in one piece: W (hi, lo), the masked
// Q K^T (forward only) and the scalars exp(cum), exp(cum_end - cum), beta of the chunk's tokens, then cum as
// a sum of two floats. The matrices are right operands of tcgen05 products without a swizzle: blocks of
// 16 x 16 of the lower triangle, by column of blocks, each as 8 x 8 core matrices of 128 contiguous bytes
// (rows 0-7: two halves of the columns, then rows 8-15). Then, for the backward pass alone, W and the masked
// Q K^T (hi, lo each) by row of blocks, for products that sum over their rows (columns 0-7: the two
// halves of the rows, then columns 8-15).
constexpr int kBlockBytes = 512;
constexpr int kWBytes = kBlocks * 2 * kBlockBytes;
constexpr int kPBytes = kBlocks * kBlockBytes;
constexpr int kScalBytes = 5 * kC * 4;
template <bool BWD>
struct Prep {
    static constexpr int W = 0, P = kWBytes, scal = BWD ? kWBytes : P + kPBytes, Wr = scal + kScalBytes, Pr = Wr + kWBytes;
    static constexpr int bytes = BWD ? Pr + kWBytes : scal + kScalBytes;
};
// block (a, b) by column of blocks: four of column 0, three of column 1, ...
__host__ __device__ constexpr int column_at(int a, int b) { return b * 4 - b * (b - 1) / 2 + a - b; }

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
// Left operand (16 x 16) from two neighbouring accumulator tiles: the same elements, converted.
__device__ __forceinline__ void split_a(const float (&t0)[4], const float (&t1)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(t0[0], t0[1], hi[0], lo[0]);
    split2(t0[2], t0[3], hi[1], lo[1]);
    split2(t1[0], t1[1], hi[2], lo[2]);
    split2(t1[2], t1[3], hi[3], lo[3]);
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
// mma.sync (550 TFLOP/s measured) because the products are 16 x 16 and depend on one another: a block stays in
// registers from one to the next. Bound by issue, about 3300 instructions per chunk and head, 16 warps per SM (shared
// memory allows 4 CTAs): 24 heads, 8 x 2048 tokens, 43 us; 80 heads, 4 x 8192, 204 us.
constexpr double kLog2e = 1.4426950408889634;
constexpr int kDl = 20;  // padded row of a diagonal block
// The fp32 products are kept up to the diagonal block: row i of block row a has 16 (a + 1) columns and a
// pad of 8 (a half warp's pairs then fall in different banks).
__device__ __forceinline__ int tri_at(int i) {
    const int a = i >> 4;
    return 16 * (4 * a * (2 * a + 4)) + (i & 15) * (16 * a + 24);
}
constexpr int kTriFloats = 16 * (24 + 40 + 56 + 72);

struct PrepWarp {
    float diag[4][16 * kDl];
    float ch[kC], cl[kC];  // log2(e) cum as a sum of two floats
    float beta[kC];
};
template <int NT>
union PrepSmem {
    struct {
        __nv_bfloat16 k[kC * NT], q[kC * NT];
    };
    struct {  // once K and Q are done with
        float kk[kTriFloats], qk[kTriFloats];
        PrepWarp w[4];
    };
};

// Right-operand fragments (hi, lo) of a 16 x 16 fp32 block in accumulator layout, rows g and g + 8 scaled.
__device__ __forceinline__ void split_b(const float (&b)[2][4], float s0, float s1, uint32_t (&h)[4], uint32_t (&l)[4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        split2(s0 * b[n][0], s0 * b[n][1], h[2 * n], l[2 * n]);
        split2(s1 * b[n][2], s1 * b[n][3], h[2 * n + 1], l[2 * n + 1]);
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

// Block (a, b) by row of blocks, hi and lo (fragments: rows 0-7, two halves of the columns, then rows 8-15).
__device__ __forceinline__ void put_rows(char *out, int a, int b, int lane, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
    uint32_t *t = reinterpret_cast<uint32_t *>(out + block_at(a, b) * kBlockBytes) + lane;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int at = 32 * ((e & 1) * 2 + (e >> 1));  // columns first
        t[at] = hi[e];
        t[at + kWBytes / 8] = lo[e];
    }
}

// Block (a, b) of W.
template <bool BWD>
__device__ __forceinline__ void put_w(char *out, int a, int b, int lane, const float (&w)[2][4]) {
    uint32_t hi[4], lo[4];  // rows 0-7: two halves of the columns, then rows 8-15
    split2(w[0][0], w[0][1], hi[0], lo[0]);
    split2(w[1][0], w[1][1], hi[1], lo[1]);
    split2(w[0][2], w[0][3], hi[2], lo[2]);
    split2(w[1][2], w[1][3], hi[3], lo[3]);
    uint32_t *t = reinterpret_cast<uint32_t *>(out + Prep<BWD>::W + column_at(a, b) * kBlockBytes) + lane;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        t[32 * e] = hi[e];
        t[32 * e + kWBytes / 8] = lo[e];
    }
    if constexpr (BWD) put_rows(out + Prep<BWD>::Wr, a, b, lane, hi, lo);
}

template <int NT, bool BWD>
__global__ void __launch_bounds__(kThr, 4)
    k_delta_prep(const __nv_bfloat16 *__restrict__ Bm, const __nv_bfloat16 *__restrict__ Cm, const __nv_bfloat16 *__restrict__ g,
                 const __nv_bfloat16 *__restrict__ beta, int64_t L, int H, int G, int N, int slices, char *__restrict__ ws,
                 int *__restrict__ clear, int nclear) {
    extern __shared__ __align__(128) char raw[];
    PrepSmem<NT> &sm = *reinterpret_cast<PrepSmem<NT> *>(raw);
    using Lay = Prep<BWD>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tg = lane & 3;
    const int64_t c = blockIdx.x, nc = gridDim.x, b = blockIdx.z, t0 = c * kC;
    const int grp = blockIdx.y / slices, slice = blockIdx.y % slices, per = H / G;
    const int h_begin = grp * per + per * slice / slices, h_end = grp * per + per * (slice + 1) / slices;
    const uint32_t ka = smem_u32(sm.k), qa = smem_u32(sm.q);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int i = tid; i < nclear; i += kThr) clear[i] = 0;
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
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < 2 * warp + 2) {
                const int r0 = tri_at(16 * warp + gr) + 8 * j + 2 * tg, r1 = tri_at(16 * warp + gr + 8) + 8 * j + 2 * tg;
                *reinterpret_cast<float2 *>(&sm.kk[r0]) = make_float2(kk[j][0], kk[j][1]);
                *reinterpret_cast<float2 *>(&sm.kk[r1]) = make_float2(kk[j][2], kk[j][3]);
                *reinterpret_cast<float2 *>(&sm.qk[r0]) = make_float2(qk[j][0], qk[j][1]);
                *reinterpret_cast<float2 *>(&sm.qk[r1]) = make_float2(qk[j][2], qk[j][3]);
            }
        }
    }
    __syncthreads();
    PrepWarp &wm = sm.w[warp];
    const bool in0 = t0 + 2 * lane < L, in1 = t0 + 2 * lane + 1 < L;  // 2 tokens per lane
    const auto token = [&](const __nv_bfloat16 *src, int h, int o) {
        return (o ? in1 : in0) && h < h_end ? to_f32(src[(b * L + t0 + 2 * lane + o) * H + h]) : 0.f;
    };
    float next[4] = {token(g, h_begin + warp, 0), token(g, h_begin + warp, 1), token(beta, h_begin + warp, 0), token(beta, h_begin + warp, 1)};
    for (int h = h_begin + warp; h < h_end; h += 4) {
        char *out = ws + ((b * H + h) * nc + c) * (int64_t)Lay::bytes;
        {  // cumulated log decay: 2 tokens per lane, fp64
            const double g0 = clamp_log_decay(next[0]), g1 = clamp_log_decay(next[1]);
            const float b0 = next[2], b1 = next[3];
            next[0] = token(g, h + 4, 0), next[1] = token(g, h + 4, 1), next[2] = token(beta, h + 4, 0), next[3] = token(beta, h + 4, 1);
            double sum = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double total = __shfl_sync(0xffffffffu, sum, 31), first = sum - g1;
            const float f0 = (float)first, f1 = (float)sum, l0 = (float)(first - (double)f0), l1 = (float)(sum - (double)f1);
            const double e0 = kLog2e * first, e1 = kLog2e * sum;
            const float2 eh = make_float2((float)e0, (float)e1);
            reinterpret_cast<float2 *>(wm.ch)[lane] = eh;
            reinterpret_cast<float2 *>(wm.cl)[lane] = make_float2((float)(e0 - (double)eh.x), (float)(e1 - (double)eh.y));
            reinterpret_cast<float2 *>(wm.beta)[lane] = make_float2(b0, b1);
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
            const float ih[2] = {wm.ch[16 * a + gr], wm.ch[16 * a + gr + 8]}, il[2] = {wm.cl[16 * a + gr], wm.cl[16 * a + gr + 8]};
            const float2 minus = make_float2(-1.f, -1.f), one = make_float2(1.f, 1.f);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int j = 16 * cc + 8 * n + 2 * tg;
                const float2 jh = *reinterpret_cast<const float2 *>(&wm.ch[j]), jl = *reinterpret_cast<const float2 *>(&wm.cl[j]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = 16 * a + gr + 8 * r;
                    const int at = tri_at(i) + j;
                    // (h_i - h_j) + (l_i - l_j): the difference of the large parts first
                    const float2 d = fma2(one, fma2(jh, minus, make_float2(ih[r], ih[r])), fma2(jl, minus, make_float2(il[r], il[r])));
                    const float2 e = make_float2(ex2(d.x), ex2(d.y));
                    float2 kk = mul2(e, *reinterpret_cast<const float2 *>(&sm.kk[at]));
                    float2 qk = mul2(e, *reinterpret_cast<const float2 *>(&sm.qk[at]));
                    if (a == cc) {
                        kk.x = j < i ? kk.x : 0.f, kk.y = j + 1 < i ? kk.y : 0.f;
                        qk.x = j <= i ? qk.x : 0.f, qk.y = j + 1 <= i ? qk.y : 0.f;
                    }
                    m[n][2 * r] = kk.x, m[n][2 * r + 1] = kk.y;
                    p[n][2 * r] = qk.x, p[n][2 * r + 1] = qk.y;
                }
            }
            if constexpr (BWD) {
                uint32_t ph[4], pl[4];
                split2(p[0][0], p[0][1], ph[0], pl[0]);
                split2(p[1][0], p[1][1], ph[1], pl[1]);
                split2(p[0][2], p[0][3], ph[2], pl[2]);
                split2(p[1][2], p[1][3], ph[3], pl[3]);
                put_rows(out + Lay::Pr, a, cc, lane, ph, pl);
            } else {
                uint32_t *o = reinterpret_cast<uint32_t *>(out + Lay::P + column_at(a, cc) * kBlockBytes) + lane;
                o[0] = pack_bf16(p[0][0], p[0][1]), o[32] = pack_bf16(p[1][0], p[1][1]);
                o[64] = pack_bf16(p[0][2], p[0][3]), o[96] = pack_bf16(p[1][2], p[1][3]);
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
            put_w<BWD>(out, a, a, lane, d);
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
                put_w<BWD>(out, a, bb, lane, w);
                if (a < 3) split_b(w, s0, s1, bh[block_at(a, bb)], bl[block_at(a, bb)]);
            }
        }
        __syncwarp();
    }
}

template <int NT, bool BWD>
cudaError_t prep_launch(const DeltaProblem &p, char *ws, int *clear, int nclear, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const int64_t nc = (p.L + kC - 1) / kC, units = nc * p.G * p.B;
    const int per = (int)(p.H / p.G);
    // a CTA walks all heads of a group while that leaves 4 CTAs (what fits) for every SM, and
    // four heads at least, one per warp
    const int64_t fit = (int64_t)sm_count() * 4;
    int slices = units >= fit ? 1 : (int)((fit + units - 1) / units);
    if (slices > (per + 3) / 4) slices = (per + 3) / 4;
    cudaError_t e;
    constexpr int smem = sizeof(PrepSmem<NT>);
    if ((e = cudaFuncSetAttribute(k_delta_prep<NT, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
    dim3 grid((unsigned)nc, (unsigned)(p.G * slices), (unsigned)p.B);
    k_delta_prep<NT, BWD><<<grid, kThr, smem, s>>>(static_cast<const bf *>(p.Bm), static_cast<const bf *>(p.Cm),
                                                   static_cast<const bf *>(p.g), static_cast<const bf *>(p.beta), p.L,
                                                   (int)p.H, (int)p.G, (int)p.N, slices, ws, clear, nclear);
    return cudaGetLastError();
}

// The workspace begins with the status word of the bounded waits and, 256 bytes on, the chain's counters,
// a CTA each; k_delta_prep clears both.
size_t head_bytes(const DeltaProblem &p, bool backward) {
    return kWsAlign + align_up((size_t)delta_tc_grid(p, backward) * sizeof(int), kWsAlign);
}

template <int NT>
cudaError_t fwd_launch(const DeltaProblem &p, char *ws, cudaStream_t s) {
    using L = Prep<false>;
    int *status = reinterpret_cast<int *>(ws);
    const size_t at = head_bytes(p, false);
    char *prep = ws + at + align_up(delta_tc_hand_bytes(p, false), kWsAlign);
    const cudaError_t e = prep_launch<NT, false>(p, prep, status, (int)(at / sizeof(int)), s);
    return e ? e
             : delta_tc_fwd(p, DeltaChain{prep, L::bytes, L::scal, 0, status, status + kWsAlign / sizeof(int),
                                          reinterpret_cast<float *>(ws + at), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr},
                            s);
}

// Workspace of the backward pass, as byte offsets.
struct BwdLayout {
    size_t hand, prep, states, cots, err, u, z, z_lo, dB, dC, total;
};
// Short sequences keep err and z to 2^-16 and sum over the state rows in fp32 (k_delta_grads in ssd_delta.cu, whose
// segment they fit): where dB, dC, dg and dbeta are made of few numbers, these can be small against the terms that
// cancel in them, and bf16 operands (2^-9) then show. Drawn cases with an output off by more than 3 * 2^-8 on bf16 operands, of 150
// each: 1 token of 1, 4, 16 heads 32, 13, 8; 2 tokens 14, 2, 2; 8 tokens 3, 0, 0; 32 tokens none (beyond 2^-8.6: 9, 6, 1); in fp32
// none (5.8e-3 at most). It costs 72 us against 47 (24 heads of 64 x 128, 1 token), and 427 against 183 (16 x 80 heads,
// 8 tokens, where it is not taken).
bool in_parts(const DeltaProblem &p) { return p.L < 4 || (p.L <= kSeg && p.B * p.H < 16); }
BwdLayout bwd_layout(const DeltaProblem &p) {
    const size_t chunks = (size_t)(p.B * p.H) * (size_t)((p.L + kC - 1) / kC);
    const size_t rows = (size_t)(p.B * p.L * p.H * p.P) * 2;
    const int slices = delta_grads_slices(p);
    const size_t part = in_parts(p) ? (size_t)(p.B * p.L * p.H * p.N) * 4
                        : slices > 1 ? (size_t)(p.B * p.L * p.G * slices * p.N) * 4 : 0;
    const size_t state = in_parts(p) ? 0 : chunks * (size_t)(p.P * p.N) * 2;
    BwdLayout l{};
    size_t at = head_bytes(p, true);
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, kWsAlign);
        return here;
    };
    l.hand = take(delta_tc_hand_bytes(p, true));
    l.prep = take(chunks * Prep<true>::bytes);
    l.states = take(state);
    l.cots = take(state);
    l.err = take(rows);
    l.u = take(rows);
    l.z = take(rows);
    l.z_lo = take(in_parts(p) ? rows : 0);
    l.dB = take(part);
    l.dC = take(part);
    l.total = at;
    return l;
}

template <int NT>
cudaError_t bwd_launch(const DeltaProblem &p, const DeltaGrads &gr, char *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const BwdLayout l = bwd_layout(p);
    bf *states = reinterpret_cast<bf *>(ws + l.states), *cots = reinterpret_cast<bf *>(ws + l.cots);
    bf *err = reinterpret_cast<bf *>(ws + l.err), *u = reinterpret_cast<bf *>(ws + l.u), *z = reinterpret_cast<bf *>(ws + l.z);
    float *dB = reinterpret_cast<float *>(ws + l.dB), *dC = reinterpret_cast<float *>(ws + l.dC);
    const char *prep = ws + l.prep;
    using Lay = Prep<true>;
    int *status = reinterpret_cast<int *>(ws);
    cudaError_t e = prep_launch<NT, true>(p, ws + l.prep, status, (int)(head_bytes(p, true) / sizeof(int)), s);
    const DeltaChain ch{prep, Lay::bytes, Lay::scal, Lay::Wr, status, status + kWsAlign / sizeof(int),
                        reinterpret_cast<float *>(ws + l.hand), states, err, u, cots, z, in_parts(p) ? ws + l.z_lo : nullptr};
    if (!e) e = delta_tc_bwd(p, gr, ch, s);
    if (in_parts(p)) {
        if (!e) e = delta_short_grads(p, gr, DeltaParts{err, u, z, ch.z_lo}, dB, dC, s);
        return e ? e : delta_group_sum_launch(p, dB, dC, gr.dBm, gr.dCm, s);
    }
    if (!e) e = delta_grads(p, gr, ch, dB, dC, s);
    const int slices = delta_grads_slices(p);
    if (e || slices == 1) return e;
    DeltaProblem q = p;  // "heads" of the sum: the slices
    q.H = p.G * slices;
    return delta_group_sum_launch(q, dB, dC, gr.dBm, gr.dCm, s);
}

// ---------------------------------------------------------------------------------------------
// TMA takes rows of 16-byte multiples. Other headdims and dstates run on copies with zero rows and columns added
// up to the next multiple of 8, which leave the rest as it is; the outputs are copied back. Backward pass of 48 heads of
// 243 x 34, 3602 tokens: 72 + 52 us of copies (an element per lane: 128 + 118) in 630, where the general path takes 4470.
struct Repack {
    const void *src;
    void *dst;                   // [outer][rows_out][out] from [outer][rows_in][in]
    int64_t outer;
    int rows_in, rows_out, in, out;
    int bytes;  // of an element
};
struct Repacks {
    Repack r[6];
    int n = 0;
    void add(const void *src, void *dst, int64_t outer, int64_t rows_in, int64_t rows_out, int64_t in, int64_t out, int bytes) {
        if (src && dst) r[n++] = Repack{src, dst, outer, (int)rows_in, (int)rows_out, (int)in, (int)out, bytes};
    }
};
// grid.y: which copy; a warp per row of the destination
template <typename E>
__device__ __forceinline__ void repack_rows(const Repack &c) {
    const E *src = static_cast<const E *>(c.src);
    E *dst = static_cast<E *>(c.dst);
    const int lane = threadIdx.x & 31;
    const int64_t rows = c.outer * c.rows_out;
    for (int64_t r = (int64_t)blockIdx.x * (kThr / 32) + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * (kThr / 32)) {
        const int64_t o = c.rows_out == 1 ? r : r / c.rows_out;
        const int i = (int)(r - o * c.rows_out), in = i < c.rows_in ? c.in : 0;
        const E *from = src + (o * c.rows_in + i) * c.in;
        E *to = dst + r * c.out;
        for (int j0 = lane; j0 < c.out; j0 += 128) {  // four loads, then four stores
            E v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = j0 + 32 * e < in ? from[j0 + 32 * e] : E(0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + 32 * e < c.out) to[j0 + 32 * e] = v[e];
        }
    }
}
__global__ void __launch_bounds__(kThr) k_delta_repack(const __grid_constant__ Repacks c) {
    const Repack &r = c.r[blockIdx.y];
    if (r.bytes == 2) repack_rows<uint16_t>(r);
    else repack_rows<float>(r);
}
cudaError_t repack(const Repacks &c, cudaStream_t s) {
    k_delta_repack<<<dim3((unsigned)(sm_count() * 8), (unsigned)c.n), kThr, 0, s>>>(c);
    return cudaGetLastError();
}

bool whole(const DeltaProblem &p) { return p.P % 8 == 0 && p.N % 8 == 0; }
DeltaProblem padded(const DeltaProblem &p) {
    DeltaProblem q = p;
    q.P = (p.P + 7) / 8 * 8, q.N = (p.N + 7) / 8 * 8;
    return q;
}
// Byte offsets of the copies behind the workspace of the padded problem: headdim rows (x, then y, or dy and dx),
// dstate rows (B, C, and their gradients), states.
struct Copies {
    size_t rows, cols, states, row, col, state, total;
};
Copies copies_of(const DeltaProblem &q, size_t at, bool backward) {
    Copies c{};
    c.row = align_up((size_t)(q.B * q.L * q.H * q.P) * 2, kWsAlign);
    c.col = align_up((size_t)(q.B * q.L * q.G * q.N) * 2, kWsAlign);
    c.state = align_up((size_t)(q.B * q.H * q.P * q.N) * 4, kWsAlign);
    c.rows = align_up(at, kWsAlign);
    c.cols = c.rows + (backward ? 3 : 2) * c.row;
    c.states = c.cols + (backward ? 4 : 2) * c.col;
    c.total = c.states + (backward ? 3 : 2) * c.state;
    return c;
}

size_t fwd_bytes(const DeltaProblem &p) {
    return head_bytes(p, false) + align_up(delta_tc_hand_bytes(p, false), kWsAlign) +
           (size_t)(p.B * p.H) * (size_t)((p.L + kC - 1) / kC) * Prep<false>::bytes;
}
cudaError_t fwd_of(const DeltaProblem &p, char *ws, cudaStream_t s) {
    return p.N <= 64 ? fwd_launch<64>(p, ws, s) : fwd_launch<128>(p, ws, s);
}
cudaError_t bwd_of(const DeltaProblem &p, const DeltaGrads &g, char *ws, cudaStream_t s) {
    return p.N <= 64 ? bwd_launch<64>(p, g, ws, s) : bwd_launch<128>(p, g, ws, s);
}

}  // namespace

// The sequential kernel takes as long as its token chain (0.2 us a token and CTA; n CTAs of 16 rows), this
// path at least two launches and a chunk of 64: 24 bf16 heads of 64 x 128, one sequence (n = 96), L = 96: 25.7 against
// 30.7 us here, 192: 43.0 against 33.8; four (n = 384), 24: 22.5 against 28.7, 48: 33.0 against 28.7; eight,
// 16: 25.9 against 28.6, 24: 36.1 against 28.6; 32 sequences of 80 heads, 2: 143 against 127. Copies of odd sizes cost two
// launches more. The backward pass gains at every length (8 tokens of 24 heads: 80 against 54 us).
bool delta_mma_supported(const DeltaProblem &p, bool backward) {
    const int64_t sms = sm_count(), per_sm = (p.B * p.H * ((p.P + 15) / 16) + sms - 1) / sms, least = whole(p) ? 128 : 256;
    if (!backward && p.L < least && p.L * per_sm < least) return false;
    // Below 8 rows or columns a padded tile is mostly zeros, and an output of few numbers can be small against the terms
    // that cancel in it, which are kept to 2^-17: fp32 there.
    if (p.P < 8 || p.N < 8) return false;
    return p.dtype == SSD_BF16 && p.N <= 128 && p.L < (1ll << 31) && p.B * p.H * ((p.L + kC - 1) / kC) < (1ll << 31);
}

size_t delta_mma_fwd_workspace_bytes(const DeltaProblem &p) {
    if (whole(p)) return fwd_bytes(p);
    const DeltaProblem q = padded(p);
    return copies_of(q, fwd_bytes(q), false).total;
}
int delta_mma_fwd_kernels(const DeltaProblem &p) { return whole(p) ? 2 : 4; }

cudaError_t delta_mma_fwd(const DeltaProblem &p, void *ws, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    if (whole(p)) return fwd_of(p, w, s);
    DeltaProblem q = padded(p);
    const Copies c = copies_of(q, fwd_bytes(q), false);
    const int64_t rows = p.B * p.L * p.H, cols = p.B * p.L * p.G, heads = p.B * p.H;
    Repacks in, out;
    in.add(p.x, w + c.rows, rows, 1, 1, p.P, q.P, 2);
    in.add(p.Bm, w + c.cols, cols, 1, 1, p.N, q.N, 2);
    in.add(p.Cm, w + c.cols + c.col, cols, 1, 1, p.N, q.N, 2);
    in.add(p.h0, w + c.states, heads, p.P, q.P, p.N, q.N, 4);
    q.x = w + c.rows, q.Bm = w + c.cols, q.Cm = w + c.cols + c.col, q.y = w + c.rows + c.row;
    if (p.h0) q.h0 = reinterpret_cast<float *>(w + c.states);
    if (p.h_final) q.h_final = reinterpret_cast<float *>(w + c.states + c.state);
    out.add(q.y, p.y, rows, 1, 1, q.P, p.P, 2);
    out.add(q.h_final, p.h_final, heads, q.P, p.P, q.N, p.N, 4);
    cudaError_t e = repack(in, s);
    if (!e) e = fwd_of(q, w, s);
    return e ? e : repack(out, s);
}

size_t delta_mma_bwd_workspace_bytes(const DeltaProblem &p) {
    if (whole(p)) return bwd_layout(p).total;
    const DeltaProblem q = padded(p);
    return copies_of(q, bwd_layout(q).total, true).total;
}
int delta_mma_bwd_kernels(const DeltaProblem &p) {
    return (in_parts(p) || delta_grads_slices(p) > 1 ? 4 : 3) + (whole(p) ? 0 : 2);
}

cudaError_t delta_mma_bwd(const DeltaProblem &p, const DeltaGrads &g, void *ws, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    if (whole(p)) return bwd_of(p, g, w, s);
    DeltaProblem q = padded(p);
    DeltaGrads r = g;
    const Copies c = copies_of(q, bwd_layout(q).total, true);
    const int64_t rows = p.B * p.L * p.H, cols = p.B * p.L * p.G, heads = p.B * p.H;
    const auto state = [&](int i) { return reinterpret_cast<float *>(w + c.states + i * c.state); };
    Repacks in, out;
    in.add(p.x, w + c.rows, rows, 1, 1, p.P, q.P, 2);
    in.add(g.dy, w + c.rows + c.row, rows, 1, 1, p.P, q.P, 2);
    in.add(p.Bm, w + c.cols, cols, 1, 1, p.N, q.N, 2);
    in.add(p.Cm, w + c.cols + c.col, cols, 1, 1, p.N, q.N, 2);
    in.add(p.h0, state(0), heads, p.P, q.P, p.N, q.N, 4);
    in.add(g.dh_final, state(1), heads, p.P, q.P, p.N, q.N, 4);
    q.x = w + c.rows, r.dy = w + c.rows + c.row, r.dx = w + c.rows + 2 * c.row;
    q.Bm = w + c.cols, q.Cm = w + c.cols + c.col, r.dBm = w + c.cols + 2 * c.col, r.dCm = w + c.cols + 3 * c.col;
    if (p.h0) q.h0 = state(0);
    if (g.dh_final) r.dh_final = state(1);
    if (g.dh0) r.dh0 = state(2);
    out.add(r.dx, g.dx, rows, 1, 1, q.P, p.P, 2);
    out.add(r.dBm, g.dBm, cols, 1, 1, q.N, p.N, 2);
    out.add(r.dCm, g.dCm, cols, 1, 1, q.N, p.N, 2);
    out.add(r.dh0, g.dh0, heads, q.P, p.P, q.N, p.N, 4);
    cudaError_t e = repack(in, s);
    if (!e) e = bwd_of(q, r, w, s);
    return e ? e : repack(out, s);
}

}  // namespace ssd
