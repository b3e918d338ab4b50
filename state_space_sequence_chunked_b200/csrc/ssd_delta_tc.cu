// The gated delta rule's chain over chunks on tcgen05 tensor cores (see ssd_delta_mma.cu for the
// chunked form and k_delta_prep, whose W, masked Q K^T and scalars this kernel reads). A CTA holds 128
// state rows for the whole sequence: one head's, or 64 of each of two neighbouring heads of a group
// (PAIR), which share the K and Q tiles. Rows are the TMEM lanes throughout and tokens or state
// columns the TMEM columns, so that every product takes its left operand from TMEM, where the warps
// that form it write it, and its right operand from a tile in shared memory that is loaded once per
// chunk: nothing of the state passes through shared memory.
//
//   per chunk of 64 tokens   left (TMEM)             right (shared memory)          into (TMEM)
//   R0 = S K^T               S hi, lo  [128 x N]     K  [64 x N], K-major           R   64 columns
//   Yq = S Q^T               S hi                    Q  [64 x N], K-major           Y   64
//   E  = (beta R) W^T        beta R hi, lo           W hi, lo [64 x 64], K-major    R   (over R0)
//   S += (ek u)^T K          ek u hi, lo             K, columns contiguous          S   N, fp32
//   Y  = eg Yq + u P^T       u hi, lo                P  [64 x 64]                   Y
// with R = X - eg R0, err = R + E, u = beta err, eg = exp(cum), ek = exp(cum_end - cum). W and P differ by
// head, so in a PAIR the left operand of their products is 128 tokens wide, each head's rows holding
// zeros in the other's 64. W and P are lower triangular: a step of 16 tokens j multiplies only the
// tokens i from its own block on (N = 64, 48, 32, 16).
//
// Warps (512 threads): 0 loads (TMA), 1 issues the products, 2-3 unpack W and P from fragments into
// swizzled tiles, 4-11 (T) form R, u and the state's operands (two warps per 32 lanes, half of the
// columns each), 12-15 (O) scale Yq and write Y out. TMEM, 512 columns: S 128, S hi 64, S lo 64 (later
// ek u), R 64, Y 64, beta R then u 2 x 64.
//
// What bounds it: the chain of a chunk, S -> R -> u -> S, each link a product (0.1-0.25 us) and a pass of
// the T warps over its result (0.25-0.35 us).
//
// kStore is the backward pass's recomputation: no Y, but the state entering each chunk, err and u in bf16.
//
// Every wait is bounded (tc_ptx.cuh); one that runs out sets bit 0 of the workspace's status word.
#include <algorithm>

#include "ssd_delta.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 512;
constexpr int kPanel = kC * 128;  // bytes of 64 rows of 64 bf16
constexpr int kTmS = 0, kTmHi = 128, kTmLo = 192, kTmR = 256, kTmY = 320, kTmA = 384, kTmAl = 448;
constexpr int kEk = kTmLo, kEkl = kTmLo + 32;  // ek u over S lo

template <int NT, bool PAIR, bool kStore>
struct Lay {
    static constexpr int HB = PAIR ? 2 : 1;
    static constexpr int k = 0, kBytes = NT / 64 * kPanel;
    static constexpr int q = k + kBytes, x = q + (kStore ? 0 : kBytes), w = x + 2 * kPanel;
    static constexpr int p = w + 2 * HB * kPanel;  // W hi, lo per head, then P per head
    static constexpr int stage = p + (kStore ? 0 : HB * kPanel);
    static constexpr int out = 2 * stage;                     // O warps' staging, 4 KB each (kStore: err and u)
    static constexpr int scal = out + (kStore ? 2 : 1) * 4 * 4096;  // [2 stages][HB][3][64] floats
    static constexpr int bar = scal + 2 * HB * 3 * kC * 4;
    static constexpr int bytes = bar + 256;
    // what the loader's barrier counts per chunk
    static constexpr int tx = kBytes + (kStore ? 0 : kBytes) + 2 * kPanel + HB * 3 * kC * 4;
};

struct ChainArgs {
    const float *h0;
    const char *prep;
    int64_t prep_bytes;  // per chunk and head
    int scal_at, p_at;
    int64_t L;
    int H, P, G, N;
    float *h_final;
    __nv_bfloat16 *states;
    int *status;
    int wait_us;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// hi + lo parts of a pair of fp32 values (lo: what hi leaves, rounded: 2^-18 of the value at worst)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
}

template <int NT, bool PAIR, bool kStore>
__global__ void __launch_bounds__(kThreads, 1)
    k_delta_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_o0,
               const __grid_constant__ CUtensorMap tm_o1, const ChainArgs a) {
    using Z = Lay<NT, PAIR, kStore>;
    constexpr int HB = Z::HB;
    extern __shared__ __align__(1024) unsigned char sm[];
    if ((smem_u32(sm) & 1023u) != 0) {  // the swizzled layouts need 1024-byte alignment
        if (threadIdx.x == 0) atomicOr(a.status, 2);
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Z::bar);
    uint64_t *full = bar;        // [2] K, Q, x and the scalars of the stage landed
    uint64_t *wrdy = bar + 2;    // [2] W and P unpacked (2 warps)
    uint64_t *sfree = bar + 4;   // [2] the stage's readers are done
    uint64_t *rdyR = bar + 6, *rdyE = bar + 7, *rdyS = bar + 8, *rdyQ = bar + 9, *rdyY = bar + 10;  // products done
    uint64_t *sb = bar + 11;     // the state's operands written (T)
    uint64_t *ab = bar + 12;     // beta R written (T)
    uint64_t *ub = bar + 13;     // u and ek u written (T)
    uint64_t *ys = bar + 14;     // Yq scaled (O)
    uint64_t *ofree = bar + 15;  // Y (kStore: err and u) read (O)
    uint64_t *fin = bar + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 17);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bar + 18);
    int *status = a.status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * HB, grp = h / (a.H / a.G), b = blockIdx.z;
    const int pc = PAIR ? 0 : blockIdx.x * 128;
    const int nc = (int)((a.L + kC - 1) / kC);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&wrdy[i], 2);
            mbar_init(&sfree[i], kStore ? 9 : 13);  // the products, 8 T warps, 4 O warps
        }
        mbar_init(rdyR, 1);
        mbar_init(rdyE, 1);
        mbar_init(rdyS, 1);
        mbar_init(rdyQ, 1);
        mbar_init(rdyY, 1);
        mbar_init(sb, 8);
        mbar_init(ab, 8);
        mbar_init(ub, 8);
        mbar_init(ys, 4);
        mbar_init(ofree, 4);
        mbar_init(fin, 1);
        abort_flag[0] = 0;
        abort_flag[1] = a.wait_us;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const auto scal_of = [&](int k, int e) { return reinterpret_cast<float *>(sm + Z::scal) + (k * HB + e) * 3 * kC; };
    const auto prep_of = [&](int c, int e) { return a.prep + (((int64_t)b * a.H + h + e) * nc + c) * a.prep_bytes; };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
            int c = 0;
            for (; c < nc; ++c) {
                const int k = c & 1;
                if (c >= 2 && !wait_phase(&sfree[k], (uint32_t)((c - 2) >> 1) & 1u, abort_flag, status)) break;
                unsigned char *st = sm + k * Z::stage;
                mbar_arrive_tx(&full[k], Z::tx);
                for (int pn = 0; pn < NT / 64; ++pn)
                    tma_load_4d_hint(st + Z::k + pn * kPanel, &tm_k, &full[k], 64 * pn, grp, c * kC, b, keep);
                for (int pn = 0; pn < 2; ++pn)
                    tma_load_4d_hint(st + Z::x + pn * kPanel, &tm_x, &full[k], PAIR ? 0 : pc + 64 * pn, PAIR ? h + pn : h, c * kC, b,
                                     stream);
                for (int e = 0; e < HB; ++e) bulk_load(scal_of(k, e), prep_of(c, e) + a.scal_at, 3 * kC * 4, &full[k]);
                if constexpr (!kStore)
                    for (int pn = 0; pn < NT / 64; ++pn)
                        tma_load_4d_hint(st + Z::q + pn * kPanel, &tm_q, &full[k], 64 * pn, grp, c * kC, b, keep);
            }
            // loads in flight land before the CTA exits
            for (int i = 1; i <= 2; ++i) {
                if (c - i < 0) continue;
                const unsigned long long w0 = now_ns();
                while (!mbar_try(&full[(c - i) & 1], (uint32_t)((c - i) >> 1) & 1u) && now_ns() - w0 < kWaitNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        if (lane == 0) {
            constexpr uint32_t id_ks = idesc(128, 64, false, false), id_s = idesc(128, NT, false, true);
            for (int c = 0; c < nc; ++c) {
                const int k = c & 1;
                const uint32_t par = (uint32_t)c & 1u;
                const uint32_t st = smem_u32(sm + k * Z::stage);
                if (!wait_phase(&full[k], (uint32_t)(c >> 1) & 1u, abort_flag, status)) break;
                if (!wait_phase(sb, par, abort_flag, status)) break;
                tc_fence_after();
                const uint64_t kd = sdesc(st + Z::k, 16, 1024);
#pragma unroll 1
                for (int kk = 0; kk < NT / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4);
                    mma_ts(tmem + kTmR, tmem + kTmLo + 8 * kk, kd + off, id_ks, kk > 0);
                    mma_ts(tmem + kTmR, tmem + kTmHi + 8 * kk, kd + off, id_ks, 1);
                }
                mma_commit(rdyR);
                if constexpr (!kStore) {
                    if (c > 0 && !wait_phase(ofree, par ^ 1u, abort_flag, status)) break;
                    tc_fence_after();
                    const uint64_t qd = sdesc(st + Z::q, 16, 1024);
#pragma unroll 1
                    for (int kk = 0; kk < NT / 16; ++kk)
                        mma_ts(tmem + kTmY, tmem + kTmHi + 8 * kk, qd + (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), id_ks,
                               kk > 0);
                    mma_commit(rdyQ);
                }
                // B rows from 16 i on, columns 16 i .. 16 i + 15, of a 64 x 64 tile
                const auto tri = [&](uint32_t d, uint32_t left, uint32_t tile, uint32_t acc) {
                    const uint64_t td = sdesc(tile, 16, 1024);
#pragma unroll 1
                    for (int i = 0; i < 4; ++i)
                        mma_ts(d + 16 * i, left + 8 * i, td + (uint64_t)((2048 * i + 32 * i) >> 4), idesc(128, 64 - 16 * i, false, false),
                               i > 0 ? 1u : acc);
                };
                if (!wait_phase(&wrdy[k], (uint32_t)(c >> 1) & 1u, abort_flag, status)) break;
                if (!wait_phase(ab, par, abort_flag, status)) break;
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < HB; ++e) {
                    const uint32_t wh = st + Z::w + 2 * e * kPanel;
                    tri(tmem + kTmR, tmem + kTmAl + 32 * e, wh, e);
                    tri(tmem + kTmR, tmem + kTmA + 32 * e, wh + kPanel, 1);
                    tri(tmem + kTmR, tmem + kTmA + 32 * e, wh, 1);
                }
                mma_commit(rdyE);
                if (!wait_phase(ub, par, abort_flag, status)) break;
                tc_fence_after();
                const uint64_t ks = sdesc(st + Z::k, kPanel, 1024);
#pragma unroll 1
                for (int kk = 0; kk < 4; ++kk) {
                    mma_ts(tmem + kTmS, tmem + kEkl + 8 * kk, ks + 128 * kk, id_s, 1);
                    mma_ts(tmem + kTmS, tmem + kEk + 8 * kk, ks + 128 * kk, id_s, 1);
                }
                mma_commit(rdyS);
                if constexpr (!kStore) {
                    if (!wait_phase(ys, par, abort_flag, status)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int e = 0; e < HB; ++e) {
                        tri(tmem + kTmY, tmem + kTmAl + 32 * e, st + Z::p + e * kPanel, 1);
                        tri(tmem + kTmY, tmem + kTmA + 32 * e, st + Z::p + e * kPanel, 1);
                    }
                    mma_commit(rdyY);
                }
                mma_commit(&sfree[k]);
            }
            mma_commit(fin);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------- W and P: fragments to tiles
        // A block of 16 x 16 (a, bb) is one 16-byte vector per lane: rows g and g + 8, columns 2 t (+1) and
        // 8 + 2 t (+1). Blocks go round the two warps; 10 of them are in registers while the stage is waited for.
        const int g = lane >> 2, t = lane & 3;
        constexpr int per_head = kStore ? 20 : 30, total = HB * per_head, mine = total / 2;  // 10, 15, 20 or 30
        constexpr int batch = mine % 10 == 0 ? 10 : 15;
        const auto src = [&](int c, int i) -> const uint4 * {
            const int blk = 2 * i + (warp & 1), e = blk / per_head, r = blk % per_head;
            const char *pr = prep_of(c, e);
            return reinterpret_cast<const uint4 *>(r < 20 ? pr + r * 512 : pr + a.p_at + (r - 20) * 512) + lane;
        };
        const auto put = [&](int k, int i, uint4 v) {
            const int blk = 2 * i + (warp & 1), e = blk / per_head, r = blk % per_head;
            const int at = r < 20 ? r >> 1 : r - 20;  // W: hi and lo of a block follow one another
            const int ai = at >= 6 ? 3 : at >= 3 ? 2 : at >= 1 ? 1 : 0, bj = at - ai * (ai + 1) / 2;
            unsigned char *tile = sm + k * Z::stage + (r < 20 ? Z::w + (2 * e + (r & 1)) * kPanel : Z::p + e * kPanel);
            const int row = 16 * ai + g;
            *reinterpret_cast<uint32_t *>(tile + swz(row, 2 * bj) + 4 * t) = v.x;
            *reinterpret_cast<uint32_t *>(tile + swz(row, 2 * bj + 1) + 4 * t) = v.y;
            *reinterpret_cast<uint32_t *>(tile + swz(row + 8, 2 * bj) + 4 * t) = v.z;
            *reinterpret_cast<uint32_t *>(tile + swz(row + 8, 2 * bj + 1) + 4 * t) = v.w;
        };
        for (int c = 0; c < nc; ++c) {
            const int k = c & 1;
            bool ok = true;
#pragma unroll 1
            for (int i0 = 0; i0 < mine; i0 += batch) {
                uint4 v[batch];
#pragma unroll
                for (int i = 0; i < batch; ++i) v[i] = __ldg(src(c, i0 + i));
                if (i0 == 0 && c >= 2) ok = wait_warp(&sfree[k], (uint32_t)((c - 2) >> 1) & 1u, abort_flag, status);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < batch; ++i) put(k, i0 + i, v[i]);
            }
            if (!ok) break;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&wrdy[k]);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------- T: the chain's elementwise links
        const int qtr = warp & 3, half = (warp - 4) >> 2, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);  // this warp's lanes
        const int pp = (qtr & 1) * 32 + lane;                      // row within the x panel qtr >> 1
        const int p = PAIR ? pp : pc + 32 * qtr + lane;            // state row of the head
        const int64_t srow = ((int64_t)b * a.H + h + e) * a.P + p;
        constexpr int SC = NT / 2;  // state columns of this warp, from n0 on
        const int n0 = half * SC;
        if constexpr (PAIR) {  // zeros in the other head's tokens
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0;
            tmem_st16(lo_ + kTmA + 32 * (1 - e) + 16 * half, zero);
            tmem_st16(lo_ + kTmAl + 32 * (1 - e) + 16 * half, zero);
        }
        for (int c = 0; c < nc; ++c) {
            const int k = c & 1;
            const uint32_t par = (uint32_t)c & 1u;
            if (!wait_warp(&full[k], (uint32_t)(c >> 1) & 1u, abort_flag, status)) break;
            const float *eg = scal_of(k, e), *ek = eg + kC, *bt = eg + 2 * kC;
            if (c > 0) {
                if (!wait_warp(rdyS, par ^ 1u, abort_flag, status)) break;
                tc_fence_after();
            }
            {  // the state: its operands, and itself times exp(cum_end) for the product to add to
                const float gamma = eg[kC - 1];
#pragma unroll
                for (int j = 0; j < SC; j += 32) {
                    uint32_t s[32];
                    if (c > 0) {
                        tmem_ld32(lo_ + kTmS + n0 + j, s);
                        tmem_wait_ld(s);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (a.h0 && p < a.P && n0 + j + 4 * i < a.N)
                                v = *reinterpret_cast<const float4 *>(a.h0 + srow * a.N + n0 + j + 4 * i);
                            s[4 * i] = __float_as_uint(v.x), s[4 * i + 1] = __float_as_uint(v.y);
                            s[4 * i + 2] = __float_as_uint(v.z), s[4 * i + 3] = __float_as_uint(v.w);
                        }
                    }
                    uint32_t hi[16], lw[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        split2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]), hi[i], lw[i]);
                        s[2 * i] = __float_as_uint(gamma * __uint_as_float(s[2 * i]));
                        s[2 * i + 1] = __float_as_uint(gamma * __uint_as_float(s[2 * i + 1]));
                    }
                    tmem_st16(lo_ + kTmHi + (n0 + j) / 2, hi);
                    tmem_st16(lo_ + kTmLo + (n0 + j) / 2, lw);
                    uint32_t g0[16], g1[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) g0[i] = s[i], g1[i] = s[16 + i];
                    tmem_st16(lo_ + kTmS + n0 + j, g0);
                    tmem_st16(lo_ + kTmS + n0 + j + 16, g1);
                    if constexpr (kStore) {
                        if (p < a.P) {
                            __nv_bfloat16 *dst = a.states + ((((int64_t)b * a.H + h + e) * nc + c) * a.P + p) * a.N + n0 + j;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (n0 + j + 8 * i < a.N)
                                    reinterpret_cast<uint4 *>(dst)[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sb);
            }
            // R = X - eg S K^T; beta R as left operand. This warp: tokens 32 half .. + 31.
            float R[32];
            const unsigned char *xt = sm + k * Z::stage + Z::x + (qtr >> 1) * kPanel;
            if (!wait_warp(rdyR, par, abort_flag, status)) break;
            tc_fence_after();
            {
                uint32_t r[32];
                tmem_ld32(lo_ + kTmR + 32 * half, r);
                tmem_wait_ld(r);
                if constexpr (kStore) {
                    if (c > 0 && !wait_warp(ofree, par ^ 1u, abort_flag, status)) break;
                }
                uint32_t hi[16], lw[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int t = 32 * half + i;
                    const float4 g4 = *reinterpret_cast<const float4 *>(eg + t), b4 = *reinterpret_cast<const float4 *>(bt + t);
                    float xv[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        xv[v] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(xt + swz(t + v, pp >> 3) + 2 * (pp & 7)));
                    R[i] = fmaf(-g4.x, __uint_as_float(r[i]), xv[0]);
                    R[i + 1] = fmaf(-g4.y, __uint_as_float(r[i + 1]), xv[1]);
                    R[i + 2] = fmaf(-g4.z, __uint_as_float(r[i + 2]), xv[2]);
                    R[i + 3] = fmaf(-g4.w, __uint_as_float(r[i + 3]), xv[3]);
                    split2(b4.x * R[i], b4.y * R[i + 1], hi[i / 2], lw[i / 2]);
                    split2(b4.z * R[i + 2], b4.w * R[i + 3], hi[i / 2 + 1], lw[i / 2 + 1]);
                }
                tmem_st16(lo_ + kTmA + 32 * e + 16 * half, hi);
                tmem_st16(lo_ + kTmAl + 32 * e + 16 * half, lw);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ab);
            }
            // err = R + E, u = beta err, and ek u
            if (!wait_warp(rdyE, par, abort_flag, status)) break;
            tc_fence_after();
            {
                uint32_t r[32];
                tmem_ld32(lo_ + kTmR + 32 * half, r);
                tmem_wait_ld(r);
                uint32_t hi[16], lw[16], ehi[16], elw[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int t = 32 * half + i;
                    const float4 k4 = *reinterpret_cast<const float4 *>(ek + t), b4 = *reinterpret_cast<const float4 *>(bt + t);
                    float u[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) R[i + v] += __uint_as_float(r[i + v]);
                    u[0] = b4.x * R[i], u[1] = b4.y * R[i + 1], u[2] = b4.z * R[i + 2], u[3] = b4.w * R[i + 3];
                    if constexpr (kStore) {  // u and err go out rounded; no product here takes u itself
                        hi[i / 2] = pack_bf16(u[0], u[1]), hi[i / 2 + 1] = pack_bf16(u[2], u[3]);
                        lw[i / 2] = pack_bf16(R[i], R[i + 1]), lw[i / 2 + 1] = pack_bf16(R[i + 2], R[i + 3]);
                    } else {
                        split2(u[0], u[1], hi[i / 2], lw[i / 2]);
                        split2(u[2], u[3], hi[i / 2 + 1], lw[i / 2 + 1]);
                    }
                    split2(k4.x * u[0], k4.y * u[1], ehi[i / 2], elw[i / 2]);
                    split2(k4.z * u[2], k4.w * u[3], ehi[i / 2 + 1], elw[i / 2 + 1]);
                }
                if constexpr (kStore) {
                    tmem_st16(lo_ + kTmY + 16 * half, hi);
                    tmem_st16(lo_ + kTmY + 32 + 16 * half, lw);
                } else {
                    tmem_st16(lo_ + kTmA + 32 * e + 16 * half, hi);
                    tmem_st16(lo_ + kTmAl + 32 * e + 16 * half, lw);
                }
                tmem_st16(lo_ + kEk + 16 * half, ehi);
                tmem_st16(lo_ + kEkl + 16 * half, elw);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ub);
                    mbar_arrive(&sfree[k]);
                }
            }
        }
        if (a.h_final && wait_warp(rdyS, (uint32_t)(nc - 1) & 1u, abort_flag, status)) {
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < SC; j += 32) {
                uint32_t s[32];
                tmem_ld32(lo_ + kTmS + n0 + j, s);
                tmem_wait_ld(s);
                if (p < a.P)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n0 + j + 4 * i < a.N)
                            *reinterpret_cast<uint4 *>(a.h_final + srow * a.N + n0 + j + 4 * i) =
                                make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
            }
        }
    } else {
        // ------------------------------------------------------------- O: outputs, 32 state rows x 64 tokens per warp
        const int qtr = warp & 3, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);
        const int p0 = PAIR ? (qtr & 1) * 32 : pc + 32 * qtr;  // first state row of the head
        unsigned char *stage0 = sm + Z::out + qtr * 4096, *stage1 = stage0 + 4 * 4096;  // [64 tokens][32 rows]
        const uint64_t pol = policy_evict_first();
        for (int c = 0; c < nc; ++c) {
            const int k = c & 1;
            const uint32_t par = (uint32_t)c & 1u;
            uint32_t o0[32], o1[32];
            if constexpr (!kStore) {
                if (!wait_warp(&full[k], (uint32_t)(c >> 1) & 1u, abort_flag, status)) break;
                if (!wait_warp(rdyQ, par, abort_flag, status)) break;
                tc_fence_after();
                const float *eg = scal_of(k, e);
#pragma unroll 1
                for (int j = 0; j < 64; j += 16) {
                    uint32_t r[16];
                    tmem_ld16(lo_ + kTmY + j, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(eg[j + i] * __uint_as_float(r[i]));
                    tmem_st16(lo_ + kTmY + j, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ys);
                    mbar_arrive(&sfree[k]);
                }
                if (!wait_warp(rdyY, par, abort_flag, status)) break;
            } else {
                if (!wait_warp(ub, par, abort_flag, status)) break;
            }
            tc_fence_after();
            tmem_ld32(lo_ + kTmY, o0);
            tmem_wait_ld(o0);
            tmem_ld32(lo_ + kTmY + 32, o1);
            tmem_wait_ld(o1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ofree);
                bulk_wait_read();  // the staging's last store has read it
            }
            __syncwarp();
            if constexpr (kStore) {  // pairs of tokens: u in o0, err in o1
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    *reinterpret_cast<uint16_t *>(stage0 + (2 * i) * 64 + 2 * lane) = (uint16_t)(o0[i] & 0xffffu);
                    *reinterpret_cast<uint16_t *>(stage0 + (2 * i + 1) * 64 + 2 * lane) = (uint16_t)(o0[i] >> 16);
                    *reinterpret_cast<uint16_t *>(stage1 + (2 * i) * 64 + 2 * lane) = (uint16_t)(o1[i] & 0xffffu);
                    *reinterpret_cast<uint16_t *>(stage1 + (2 * i + 1) * 64 + 2 * lane) = (uint16_t)(o1[i] >> 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    reinterpret_cast<__nv_bfloat16 *>(stage0 + i * 64)[lane] = __float2bfloat16_rn(__uint_as_float(o0[i]));
                    reinterpret_cast<__nv_bfloat16 *>(stage0 + (32 + i) * 64)[lane] = __float2bfloat16_rn(__uint_as_float(o1[i]));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && p0 < a.P) {
                tma_store_4d(&tm_o0, stage0, p0, h + e, c * kC, b, pol);
                if constexpr (kStore) tma_store_4d(&tm_o1, stage1, p0, h + e, c * kC, b, pol);
                bulk_commit();
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (lane == 0) {  // every issued product has completed before TMEM is released
            const unsigned long long t0 = now_ns();
            while (!mbar_try(fin, 0) && now_ns() - t0 < kWaitNs) {
            }
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// [B, L, X, inner] bf16, boxes of 32 columns by 64 tokens, not swizzled (the O warps' staging).
bool encode_out(CUtensorMap *m, const void *base, int64_t inner, int64_t X, int64_t L, int64_t B) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)X, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)(inner * 2), (cuuint64_t)(X * inner * 2), (cuuint64_t)(L * X * inner * 2)};
    const cuuint32_t box[4] = {32, 1, (cuuint32_t)kC, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool PAIR, bool kStore>
cudaError_t launch(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    CUtensorMap tk, tq, tx, t0, t1;
    if (!encode_4d(&tk, p.Bm, p.N, p.G, p.L, p.B, kC) || !encode_4d(&tq, p.Cm, p.N, p.G, p.L, p.B, kC) ||
        !encode_4d(&tx, p.x, p.P, p.H, p.L, p.B, kC) ||
        !encode_out(&t0, kStore ? ch.u : p.y, p.P, p.H, p.L, p.B) || !encode_out(&t1, kStore ? ch.err : p.y, p.P, p.H, p.L, p.B))
        return cudaErrorInvalidValue;
    const ChainArgs a{p.h0,       ch.prep, ch.prep_bytes, ch.scal_at, ch.p_at, p.L, (int)p.H, (int)p.P, (int)p.G, (int)p.N,
                      p.h_final, static_cast<__nv_bfloat16 *>(ch.states), ch.status, wait_limit_us()};
    constexpr int smem = Lay<NT, PAIR, kStore>::bytes;
    const auto kernel = k_delta_tc<NT, PAIR, kStore>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    const dim3 grid(PAIR ? 1u : (unsigned)((p.P + 127) / 128), (unsigned)(PAIR ? p.H / 2 : p.H), (unsigned)p.B);
    kernel<<<grid, kThreads, smem, s>>>(tk, tq, tx, t0, t1, a);
    return cudaGetLastError();
}

template <int NT, bool kStore>
cudaError_t launch_pair(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    // two heads of a group side by side where each fits 64 rows: half the CTAs, and K, Q loaded once for both
    return p.P <= 64 && (p.H / p.G) % 2 == 0 ? launch<NT, true, kStore>(p, ch, s) : launch<NT, false, kStore>(p, ch, s);
}

}  // namespace

cudaError_t delta_tc_chain(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    const bool store = ch.states != nullptr;
    if (p.N <= 64) return store ? launch_pair<64, true>(p, ch, s) : launch_pair<64, false>(p, ch, s);
    return store ? launch_pair<128, true>(p, ch, s) : launch_pair<128, false>(p, ch, s);
}

}  // namespace ssd
