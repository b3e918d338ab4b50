// The gradients of the gated delta rule that sum over the rows of the state, on tcgen05, after both chains.
// Per chunk and head, with S the state entering the chunk, D the cotangent leaving it, E_ij =
// exp(cum_i - cum_j) for i >= j, eg = exp(cum), ek = exp(cum_end - cum), u = beta err, r = beta z:
//     dP = tril((dY u^T) o E),   dM = -tril((r u^T) o E, -1),
//     dQ = eg dY S + dP K,
//     dK = -eg r S + ek u D + dM K + dP^T Q + dM^T K,
//     dbeta_i = z_i.err_i,   dg_i = what passes the decay of token i:
//         sum over t >= i > j of F_tj,  F = dP o Q K^T + dM o K K^T,
//         sum over t >= i of eg_t (dY_t.S q_t - r_t.S k_t),
//         sum over t < i of U_t = ek_t u_t.D k_t,  and exp(cum_end) <D, S>.
// No sum runs across chunks, each pair of tokens enters once, in fp32, and nothing that came in goes out again (as
// in a sum from i to the end of the derivative with respect to cum): under strong decays dg shrinks with
// exp(g), and its errors with it. The pairs t >= i > j are summed in two parts, by quarters of 16 tokens: j in the quarter
// of i, from sums of a row's columns within the quarter (cols), and j in the quarters before, whole (pairs).
//
// A CTA takes a chunk of a group and walks its heads (of its slice), 64 state rows at a time. dQ and dK of
// the chunk stand in TMEM for all of them, tokens by lane (dQ in lanes 0-63, dK in 64-127), and every term is
// a product with 128 rows that adds to both or, with a panel of zeros, to dK alone:
//     [eg dY; -eg r] S,  [0; ek u] D,  [dP; dM] K,  [0; dP^T] Q,  [0; dM^T] K
// so that the CUDA cores only scale the left operands, form dP and dM out of [dY; r] u^T, and take the
// dot products of dg with [Q; K] S^T and [Q; K] D^T. Operands are rounded to bf16 once each; sums are fp32, in
// a fixed order (no atomics).
//
// Warps (640 threads): 0 loads (TMA, two stages), 1 issues the products, 2 ends a head (dg, dbeta), 4-19 the
// elementwise work, four per 32 lanes with a quarter of the columns each.
//
// Bound by the elementwise warps: 6100 cycles per head and 64 rows with the ends of a CTA, of which they work 4400 and
// the products take 2400. 24 heads of 64 x 128, 4 x 2048 tokens: 84 us, of 24 us for its bytes; the same sums
// with mma.sync, dQ and dK in registers, took 212. Issuing a step's first products before the last step's pairs,
// or waiting for fewer of them, gained nothing (87 and 93 us).
//
// Every wait is bounded (tc_ptx.cuh); one that runs out sets bit 0 of the workspace's status word.
#include "delta_tc.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kCWarps = 16, kThreads = 32 * (4 + kCWarps);
constexpr float kLog2e = 1.44269504f;
constexpr int kTmG = 0, kTmP = 128, kTmS = 192, kTmD = 256, kTmConst = 320;

struct HeadSums {
    float rows[4][128];   // eg dY.S q and -eg r.S k by quarter of the state rows: dQ-side and dK-side tokens
    float pairs[3][128];  // F's rows over the columns of a quarter
    float cols[4][kC];    // its pairs t >= i > j with j in the quarter of i, by lane quarter
    float U[4][kC];
    float dot[kCWarps / 2], db[kC];
};

template <int NT>
struct Lay {
    static constexpr int pn = NT / 64;
    static constexpr int qk = 0;                                  // [panel][Q 64 rows, K 64 rows]
    static constexpr int x1 = qk + pn * 2 * kPanel;               // [eg dY; -eg r]
    static constexpr int zero = x1 + 2 * kPanel, x2 = zero + kPanel;  // [0; ek u]
    static constexpr int dp = x2 + kPanel;                        // [dP; dM]
    static constexpr int s = 0, d = pn * kPanel, dy = 2 * pn * kPanel, r = dy + kPanel, u = r + kPanel, stage = u + kPanel;
    static constexpr int stages = dp + 2 * kPanel;
    static constexpr int scal = stages + 2 * stage;               // [2][eg, ek, beta, cum as two floats][64]
    static constexpr int sums = scal + 2 * 5 * kC * 4;
    static constexpr int bar = sums + 2 * (int)sizeof(HeadSums);
    static constexpr int bytes = bar + 256;
    static constexpr int tx = stage;
};

struct GradArgs {
    const char *prep;
    int64_t prep_bytes;
    int scal_at, nc, L, H, P, G, N, slices;
    const __nv_bfloat16 *z, *err;
    __nv_bfloat16 *dBm, *dCm, *dg, *dbeta;
    float *dB_part, *dC_part;
    int *status;
    int wait_us;
};
struct Maps {
    CUtensorMap k, q, dy, r, u, s, d;
};

__device__ __forceinline__ uint32_t scale_pair(float f, uint32_t v) {
    const float2 m = mul2(make_float2(f, f), make_float2(bf16_lo(v), bf16_hi(v)));
    return pack_bf16(m.x, m.y);
}
__device__ __forceinline__ uint4 scale8(float f, uint4 v) {
    return make_uint4(scale_pair(f, v.x), scale_pair(f, v.y), scale_pair(f, v.z), scale_pair(f, v.w));
}
// s + the products of two rows of eight, lanes of s apart
__device__ __forceinline__ float2 dot8(uint4 a, uint4 b, float2 s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s = fma2(make_float2(bf16_lo(x[i]), bf16_hi(x[i])), make_float2(bf16_lo(y[i]), bf16_hi(y[i])), s);
    return s;
}
// a TMEM row piece (16 columns) by the same columns of a bf16 row
__device__ __forceinline__ float dot16(const uint32_t (&v)[16], uint4 a, uint4 b) {
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma2(pair_of(v[2 * i], v[2 * i + 1]), make_float2(bf16_lo(x[i]), bf16_hi(x[i])), s);
    return s.x + s.y;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) k_delta_grads_tc(const __grid_constant__ Maps m, const __grid_constant__ GradArgs a) {
    using Z = Lay<NT>;
    extern __shared__ __align__(1024) unsigned char sm[];
    if ((smem_u32(sm) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(a.status, 2);
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Z::bar);
    uint64_t *full = bar, *sfree = bar + 2;      // [2] a stage's loads landed; its readers done
    uint64_t *rdyC = bar + 4, *rdyD = bar + 5;   // Q K^T and K K^T; a step's products to be read
    uint64_t *done = bar + 6, *xdone = bar + 15; // a step's products into dQ, dK; those with the scaled rows
    uint64_t *dfree = bar + 7;                   // the products read
    uint64_t *xb = bar + 8, *pb = bar + 9;       // left operands written: scaled rows; dP, dM
    uint64_t *hd = bar + 10, *hfree = bar + 12;  // [2] a head's sums written; read
    uint64_t *fin = bar + 14;
    int *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x, b = blockIdx.z, t0 = c * kC, nt = a.L - t0 < kC ? a.L - t0 : kC;
    const int grp = blockIdx.y / a.slices, slice = blockIdx.y % a.slices, per = a.H / a.G;
    const int h_begin = grp * per + per * slice / a.slices, h_end = grp * per + per * (slice + 1) / a.slices;
    const int nslab = (a.P + 63) / 64, steps = (h_end - h_begin) * nslab;
    for (int i = threadIdx.x; i < kPanel / 16; i += kThreads) reinterpret_cast<uint4 *>(sm + Z::zero)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
    constexpr int counts[16] = {1, 1, 1 + kCWarps, 1 + kCWarps, 1, 1, 1, kCWarps, kCWarps, kCWarps, kCWarps, kCWarps, 1, 1, 1, 1};
    const Setup su = set_up(bar, counts, a.wait_us, warp);
    const uint32_t tmem = su.tmem;
    volatile int *abort_flag = su.abort_flag;
    const auto stage_of = [&](int k) { return sm + Z::stages + k * Z::stage; };
    const auto scal_of = [&](int k) { return reinterpret_cast<const float *>(sm + Z::scal + k * 5 * kC * 4); };
    const auto sums_of = [&](int turn) { return reinterpret_cast<HeadSums *>(sm + Z::sums) + (turn & 1); };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t once = policy_evict_first();
            int it = 0;
            for (int h = h_begin, p = 0; it < steps; ++it, p += 64) {
                if (p >= a.P) p = 0, ++h;
                const int k = it & 1;
                if (it >= 2 && !wait_phase(&sfree[k], (uint32_t)((it - 2) >> 1) & 1u, abort_flag, status)) break;
                unsigned char *st = stage_of(k);
                mbar_arrive_tx(&full[k], Z::tx + 5 * kC * 4 + (it == 0 ? Z::pn * 2 * kPanel : 0));
                if (it == 0)
                    for (int pn = 0; pn < Z::pn; ++pn) {
                        tma_load_4d(sm + Z::qk + pn * 2 * kPanel, &m.q, &full[k], 64 * pn, grp, t0, b);
                        tma_load_4d(sm + Z::qk + pn * 2 * kPanel + kPanel, &m.k, &full[k], 64 * pn, grp, t0, b);
                    }
                const int unit = (b * a.H + h) * a.nc + c;
                bulk_load(sm + Z::scal + k * 5 * kC * 4, a.prep + (int64_t)unit * a.prep_bytes + a.scal_at, 5 * kC * 4, &full[k]);
                tma_load_4d_hint(st + Z::dy, &m.dy, &full[k], p, h, t0, b, once);
                tma_load_4d_hint(st + Z::r, &m.r, &full[k], p, h, t0, b, once);
                tma_load_4d_hint(st + Z::u, &m.u, &full[k], p, h, t0, b, once);
                for (int pn = 0; pn < Z::pn; ++pn) {
                    tma_load_4d_hint(st + Z::s + pn * kPanel, &m.s, &full[k], 64 * pn, p, unit, 0, once);
                    tma_load_4d_hint(st + Z::d + pn * kPanel, &m.d, &full[k], 64 * pn, p, unit, 0, once);
                }
            }
            drain_loads(full, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t el = elect_one(), base = smem_u32(sm);
        constexpr uint32_t id64 = idesc(128, 64, false, false);                // K-major both, N = 64
        constexpr uint32_t idn = idesc(128, NT, false, true), idt = idesc(128, NT, true, true);  // into dQ, dK
        const uint64_t qk = sdesc(base + Z::qk, 16, 1024), kr = sdesc(base + Z::qk + kPanel, 16, 1024);
        const uint64_t qn = sdesc(base + Z::qk, 2 * kPanel, 1024), kn = sdesc(base + Z::qk + kPanel, 2 * kPanel, 1024);
        const uint64_t x1 = sdesc(base + Z::x1, 16, 1024), x2 = sdesc(base + Z::zero, 16, 1024), dp = sdesc(base + Z::dp, 16, 1024);
        const uint64_t dpt = sdesc(base + Z::zero, Z::dp - Z::zero, 1024), dmt = sdesc(base + Z::zero, Z::dp + kPanel - Z::zero, 1024);
        for (int it = 0, slab = -1; it < steps; ++it) {
            if (++slab == nslab) slab = 0;
            const int k = it & 1;
            const uint32_t par = (uint32_t)it & 1u, st = base + Z::stages + k * Z::stage;
            if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
            if (it == 0) {
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < NT / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * 2 * kPanel + (kk & 3) * 32) >> 4);
                    mma_ss_el(el, tm + kTmConst, qk + off, kr + off, id64, kk > 0);
                }
                commit_el(el, rdyC);
            }
            if (it > 0 && !wait_warp(dfree, par ^ 1u, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t dyr = sdesc(st + Z::dy, 16, 1024), ur = sdesc(st + Z::u, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss_el(el, tm + kTmP, dyr + 2 * kk, ur + 2 * kk, id64, slab > 0 || kk > 0);
            const uint64_t sr = sdesc(st + Z::s, 16, 1024), dr = sdesc(st + Z::d, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < NT / 16; ++kk) {
                const uint64_t offa = (uint64_t)(((kk >> 2) * 2 * kPanel + (kk & 3) * 32) >> 4);
                const uint64_t offb = (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4);
                mma_ss_el(el, tm + kTmS, qk + offa, sr + offb, id64, kk > 0);
                mma_ss_el(el, tm + kTmD, qk + offa, dr + offb, id64, kk > 0);
            }
            commit_el(el, rdyD);
            if (!wait_warp(xb, par, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t sn = sdesc(st + Z::s, kPanel, 1024), dn = sdesc(st + Z::d, kPanel, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_ss_el(el, tm + kTmG, x1 + 2 * kk, sn + 128 * kk, idn, it > 0 || kk > 0);
                mma_ss_el(el, tm + kTmG, x2 + 2 * kk, dn + 128 * kk, idn, 1);
            }
            commit_el(el, xdone);
            if (!wait_warp(pb, par, abort_flag, status)) break;
            if (slab == nslab - 1) {
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_ss_el(el, tm + kTmG, dp + 2 * kk, kn + 128 * kk, idn, 1);
                    mma_ss_el(el, tm + kTmG, dpt + 128 * kk, qn + 128 * kk, idt, 1);
                    mma_ss_el(el, tm + kTmG, dmt + 128 * kk, kn + 128 * kk, idt, 1);
                }
            }
            commit_el(el, done);
            commit_el(el, &sfree[k]);
        }
        commit_el(el, fin);
    } else if (warp == 2) {
        // ------------------------------------------------------------- a head's end: dg and dbeta, 2 tokens per lane
        for (int turn = 0; turn < h_end - h_begin; ++turn) {
            if (!wait_warp(&hd[turn & 1], (uint32_t)(turn >> 1) & 1u, abort_flag, status)) break;
            const HeadSums &s = *sums_of(turn);
            float end = lane < kCWarps / 2 ? s.dot[lane] : 0.f;
            // from a token on: rows, pairs with columns in quarter 0, 1, 2; up to a token: U; and its own
            float after[2][4], u[2], d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                after[e][0] = d[e] = 0.f;
#pragma unroll
                for (int o = 0; o < 4; ++o) after[e][0] += s.rows[o][i] + s.rows[o][64 + i], d[e] += s.cols[o][i];
#pragma unroll
                for (int o = 0; o < 3; ++o) after[e][1 + o] = s.pairs[o][i] + s.pairs[o][64 + i];
                u[e] = (s.U[0][i] + s.U[1][i]) + (s.U[2][i] + s.U[3][i]);
            }
            const float b0 = s.db[2 * lane], b1 = s.db[2 * lane + 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&hfree[turn & 1]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) end += __shfl_xor_sync(0xffffffffu, end, o);
            float from[4], upto = u[0] + u[1];
#pragma unroll
            for (int m = 0; m < 4; ++m) from[m] = after[0][m] + after[1][m];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float v = __shfl_down_sync(0xffffffffu, from[m], o);
                    if (lane + o < 32) from[m] += v;
                }
                const float v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            upto = __shfl_up_sync(0xffffffffu, upto, 1);  // the tokens before 2 lane
            if (lane == 0) upto = 0.f;
            const int quarter = lane >> 3;
            d[0] += end + upto, d[1] += end + (upto + u[0]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float nxt = __shfl_down_sync(0xffffffffu, from[m], 1);  // from token 2 lane + 2 on
                nxt = lane < 31 ? nxt : 0.f;
                if (m <= quarter) d[0] += from[m], d[1] += after[1][m] + nxt;
            }
            const int64_t at = ((int64_t)b * a.L + t0 + 2 * lane) * a.H + h_begin + turn;
            if (2 * lane < nt) a.dg[at] = __float2bfloat16_rn(d[0]), a.dbeta[at] = __float2bfloat16_rn(b0);
            if (2 * lane + 1 < nt)
                a.dg[at + a.H] = __float2bfloat16_rn(d[1]), a.dbeta[at + a.H] = __float2bfloat16_rn(b1);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------- elementwise
        const int qtr = warp & 3, sub = (warp - 4) >> 2;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);
        const int row = 32 * qtr + lane, i = row & 63;  // lane of TMEM; its token
        const bool upper = row >= 64;                   // (warp-uniform) the rows of dK
        const int ct = (warp - 4) * 32 + lane, lt = ct >> 3, lc = ct & 7;  // and by 16-byte vector: token, vector
        float rowsum = 0.f, usum = 0.f;
        float2 dots = make_float2(0.f, 0.f), db = dots;
        // z and err of a step, one vector per thread; the next step's are asked for while this one's are used
        const int64_t zat = (((int64_t)b * a.L + t0 + lt) * a.H + h_begin) * a.P + 8 * lc;
        const __nv_bfloat16 *zp = a.z + zat, *ep = a.err + zat;
        const auto vec = [&](const __nv_bfloat16 *src, int p) {
            return lt < nt && p + 8 * lc < a.P ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
        };
        uint4 zv = vec(zp, 0), ev = vec(ep, 0);
        bool ok = true;
        for (int it = 0, turn = 0, slab = -1; it < steps; ++it) {
            const int k = it & 1;
            if (++slab == nslab) slab = 0, ++turn;
            const uint32_t par = (uint32_t)it & 1u;
            ok = false;
            if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
            const unsigned char *st = stage_of(k);
            const float *eg = scal_of(k), *ek = eg + kC, *ch = eg + 3 * kC, *cl = eg + 4 * kC;
            if (it > 0 && !wait_warp(xdone, par ^ 1u, abort_flag, status)) break;  // the last step's were read
            {
                const uint32_t at = swz(lt, lc);
                const float g = eg[lt], kf = ek[lt];
                const uint4 yv = *reinterpret_cast<const uint4 *>(st + Z::dy + at), rv = *reinterpret_cast<const uint4 *>(st + Z::r + at);
                const uint4 uv = *reinterpret_cast<const uint4 *>(st + Z::u + at);
                *reinterpret_cast<uint4 *>(sm + Z::x1 + at) = scale8(g, yv);
                *reinterpret_cast<uint4 *>(sm + Z::x1 + kPanel + at) = scale8(-g, rv);
                *reinterpret_cast<uint4 *>(sm + Z::x2 + at) = scale8(kf, uv);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(xb);
            }
            if (it == 0 && !wait_warp(rdyC, 0, abort_flag, status)) break;
            if (it > 0 && !wait_warp(done, par ^ 1u, abort_flag, status)) break;  // dP and dM were read
            if (slab == 0) {
                rowsum = usum = 0.f;
                dots = db = make_float2(0.f, 0.f);
                // the sums of the head before last have been read
                if (turn >= 2 && !wait_warp(&hfree[turn & 1], (uint32_t)((turn - 2) >> 1) & 1u, abort_flag, status)) break;
            }
            if (!wait_warp(rdyD, par, abort_flag, status)) break;
            tc_fence_after();
            HeadSums &s = *sums_of(turn);
            if (slab == nslab - 1) {  // the pairs: tokens 16 sub .. + 15 of this row
                uint32_t v[16], w[16];
                tmem_ld16(lo_ + kTmP + 16 * sub, v);
                tmem_ld16(lo_ + kTmConst + 16 * sub, w);
                tmem_wait_ld16(v);
                tmem_wait_ld16(w);
                const float ih = ch[i], il = cl[i], sign = upper ? -1.f : 1.f;
                const int last = upper ? i - 1 : i;
                const float2 minus = make_float2(-1.f, -1.f);
                float pr[16], run = 0.f;  // F's columns of the quarter before each one, in rows from its token on
                uint32_t o[8];
                if (16 * sub > (i | 31)) {  // (warp-uniform) above the diagonal
#pragma unroll
                    for (int j = 0; j < 16; ++j) pr[j] = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = 0;
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const int jj = 16 * sub + j;
                        const float4 h4 = *reinterpret_cast<const float4 *>(ch + jj), l4 = *reinterpret_cast<const float4 *>(cl + jj);
                        const float2 hj[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)};
                        const float2 lj[2] = {make_float2(l4.x, l4.y), make_float2(l4.z, l4.w)};
                        float x[4];
#pragma unroll
                        for (int n = 0; n < 4; n += 2) {
                            // log2(e) ((h_i - h_j) + (l_i - l_j)): the difference of the large parts first
                            float2 d = fma2(hj[n / 2], minus, make_float2(ih, ih));
                            d = mul2(make_float2(kLog2e, kLog2e), fma2(make_float2(1.f, 1.f), d, fma2(lj[n / 2], minus, make_float2(il, il))));
                            const float2 ex = mul2(make_float2(sign, sign), make_float2(ex2(d.x), ex2(d.y)));
                            const float2 m = mul2(ex, pair_of(v[j + n], v[j + n + 1]));
                            x[n] = jj + n <= last ? m.x : 0.f, x[n + 1] = jj + n + 1 <= last ? m.y : 0.f;
                            const float2 pq = mul2(make_float2(x[n], x[n + 1]), pair_of(w[j + n], w[j + n + 1]));
                            pr[j + n] = jj + n <= i ? run : 0.f;
                            run += pq.x;
                            pr[j + n + 1] = jj + n + 1 <= i ? run : 0.f;
                            run += pq.y;
                        }
                        o[j / 2] = pack_bf16(x[0], x[1]), o[j / 2 + 1] = pack_bf16(x[2], x[3]);
                    }
                }
                *reinterpret_cast<uint4 *>(sm + Z::dp + swz(row, 2 * sub)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(sm + Z::dp + swz(row, 2 * sub + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(pb);
                // columns: halves exchanged and added, so that lane l ends with column l >> 1
#pragma unroll
                for (int w2 = 8, x = 16; w2 >= 1; w2 >>= 1, x >>= 1)
#pragma unroll
                    for (int j = 0; j < w2; ++j) {
                        const bool up = lane & x;
                        const float send = up ? pr[j] : pr[j + w2], keep = up ? pr[j + w2] : pr[j];
                        pr[j] = keep + __shfl_xor_sync(0xffffffffu, send, x);
                    }
                pr[0] += __shfl_xor_sync(0xffffffffu, pr[0], 1);
                if ((lane & 1) == 0) s.cols[qtr][16 * sub + (lane >> 1)] = pr[0];
                if (sub < 3) s.pairs[sub][row] = run;
            } else if (lane == 0) {
                mbar_arrive(pb);
            }
            {  // dot products of dg, columns (state rows) 16 sub .. + 15 of the slab
                uint32_t v[16], w[16];
                tmem_ld16(lo_ + kTmS + 16 * sub, v);
                tmem_ld16(lo_ + kTmD + 16 * sub, w);
                tmem_wait_ld16(v);
                tmem_wait_ld16(w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dfree);
                const unsigned char *rw = st + Z::dy;  // [dY; r], 128 rows
                const float d1 = dot16(v, *reinterpret_cast<const uint4 *>(rw + swz(row, 2 * sub)),
                                       *reinterpret_cast<const uint4 *>(rw + swz(row, 2 * sub + 1)));
                if (upper) {
                    const float d2 = dot16(w, *reinterpret_cast<const uint4 *>(st + Z::u + swz(i, 2 * sub)),
                                           *reinterpret_cast<const uint4 *>(st + Z::u + swz(i, 2 * sub + 1)));
                    const float U = ek[i] * d2;
                    usum += U;
                    rowsum -= eg[i] * d1;
                } else {
                    rowsum += eg[i] * d1;
                }
            }
            // <D, S> and dbeta
            if ((qtr & 1) == 0)  // half of these warps' pairs lie above the diagonal
#pragma unroll
                for (int v = 0; v < 2 * Z::pn; ++v) {
                    const int at = (sub * 2 + (qtr >> 1)) * 32 + lane + 256 * v;
                    dots = dot8(reinterpret_cast<const uint4 *>(st + Z::s)[at], reinterpret_cast<const uint4 *>(st + Z::d)[at], dots);
                }
            db = dot8(zv, ev, db);
            if (it + 1 < steps) {
                // the next slab of the head, or the next head (rows of P, heads side by side)
                const bool more = slab + 1 < nslab;
                const int step = more ? 64 : a.P - 64 * slab;
                zp += step, ep += step;
                zv = vec(zp, more ? 64 * (slab + 1) : 0), ev = vec(ep, more ? 64 * (slab + 1) : 0);
            }
            if (slab == nslab - 1) {
                s.rows[sub][row] = rowsum;
                if (upper) s.U[sub][i] = usum;
                float ds = dots.x + dots.y, zs = db.x + db.y;
                if ((qtr & 1) == 0) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
                    if (lane == 0) s.dot[sub * 2 + (qtr >> 1)] = eg[kC - 1] * ds;
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) zs += __shfl_xor_sync(0xffffffffu, zs, o);
                if (lc == 0) s.db[lt] = zs;
                __syncwarp();
                if (lane == 0) mbar_arrive(&hd[turn & 1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[k]);
            ok = true;
        }
        if (ok && wait_warp(done, (uint32_t)(steps - 1) & 1u, abort_flag, status)) {  // dQ and dK
            tc_fence_after();
            constexpr int W = NT / 4;
            const bool live = i < nt;
            const int64_t tok = (int64_t)b * a.L + t0 + i;
#pragma unroll
            for (int j = 0; j < W; j += 16) {
                uint32_t v[16];
                tmem_ld16(lo_ + kTmG + W * sub + j, v);
                tmem_wait_ld16(v);
#pragma unroll
                for (int n = 0; n < 16; n += 8) {
                    const int col = W * sub + j + n;
                    if (!live || col >= a.N) continue;
                    const float *f = reinterpret_cast<const float *>(v + n);
                    if (a.slices == 1) {
                        __nv_bfloat16 *dst = (upper ? a.dBm : a.dCm) + (tok * a.G + grp) * a.N + col;
                        *reinterpret_cast<uint4 *>(dst) =
                            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
                    } else {
                        float *dst = (upper ? a.dB_part : a.dC_part) + (tok * gridDim.y + blockIdx.y) * a.N + col;
                        reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
                        reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
                    }
                }
            }
        }
    }
    tear_down(tmem, fin, warp, lane);
}

// [units, P, N] bf16 states, boxes of 64 columns by 64 rows, 128-byte swizzle.
bool encode_state_tiles(CUtensorMap *m, const void *base, int64_t N, int64_t P, int64_t units) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)N, (cuuint64_t)P, (cuuint64_t)units, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)(N * 2), (cuuint64_t)(P * N * 2), (cuuint64_t)(units * P * N * 2)};
    const cuuint32_t box[4] = {64, 64, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, float *dB_part, float *dC_part, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const int64_t nc = (p.L + kC - 1) / kC, units = p.B * p.H * nc;
    Maps m;
    if (!encode_4d(&m.k, p.Bm, p.N, p.G, p.L, p.B, kC) || !encode_4d(&m.q, p.Cm, p.N, p.G, p.L, p.B, kC) ||
        !encode_4d(&m.dy, g.dy, p.P, p.H, p.L, p.B, kC) || !encode_4d(&m.r, g.dx, p.P, p.H, p.L, p.B, kC) ||
        !encode_4d(&m.u, ch.u, p.P, p.H, p.L, p.B, kC) || !encode_state_tiles(&m.s, ch.states, p.N, p.P, units) ||
        !encode_state_tiles(&m.d, ch.cots, p.N, p.P, units))
        return cudaErrorInvalidValue;
    const int slices = delta_grads_slices(p);
    const GradArgs a{ch.prep, ch.prep_bytes, ch.scal_at, (int)nc, (int)p.L, (int)p.H, (int)p.P, (int)p.G, (int)p.N, slices,
                     static_cast<const bf *>(ch.z), static_cast<const bf *>(ch.err), static_cast<bf *>(g.dBm), static_cast<bf *>(g.dCm),
                     static_cast<bf *>(g.dg), static_cast<bf *>(g.dbeta), dB_part, dC_part, ch.status, wait_limit_us()};
    constexpr int smem = Lay<NT>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(k_delta_grads_tc<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    k_delta_grads_tc<NT><<<dim3((unsigned)nc, (unsigned)(p.G * slices), (unsigned)p.B), kThreads, smem, s>>>(m, a);
    return cudaGetLastError();
}

}  // namespace

// Slices of a group's heads: the number that makes (waves of CTAs on the SMs) x (heads a CTA walks)
// smallest, the fewest of them unless more save an eighth (more than one costs fp32 parts and a second
// pass).
int delta_grads_slices(const DeltaProblem &p) {
    const int64_t units = (p.L + kC - 1) / kC * p.G * p.B, per = p.H / p.G, sms = sm_count();
    int best = 1;
    int64_t cost = (units + sms - 1) / sms * per;
    for (int s = 2; s <= per && s <= 16; ++s) {
        const int64_t here = (units * s + sms - 1) / sms * ((per + s - 1) / s);
        if (here * 8 < cost * 7) cost = here, best = s;
    }
    return best;
}

cudaError_t delta_grads(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, float *dB_part, float *dC_part,
                        cudaStream_t s) {
    return p.N <= 64 ? launch<64>(p, g, ch, dB_part, dC_part, s) : launch<128>(p, g, ch, dB_part, dC_part, s);
}

}  // namespace ssd
