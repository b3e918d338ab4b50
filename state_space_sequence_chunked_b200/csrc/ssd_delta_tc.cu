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
// head, so in a PAIR each of their products is issued once per head and writes that head's 64 lanes alone: a head's
// values that are not finite stay its own. W and P are lower triangular: a step of 16 tokens j
// multiplies only the tokens i from its own block on (N = 64, 48, 32, 16). (Within such a step the zeros above the
// diagonal are multiplied: a value that is not finite reaches the tokens before it in its block of 16.)
//
// Warps (768 threads): 0 loads (TMA), 1 issues the products, 4-19 (T) form R, u and the state's operands (four
// warps per 32 lanes, a quarter of the columns each), 20-23 (O) scale Yq and write Y out; in the forward
// chain 2-3 are idle (a T or O warp's TMEM lanes are those of its number modulo 4). TMEM, 512 columns: S 128,
// S hi 64, S lo 64 (later ek u), R 64, Y 64, beta R then u 32 + 32 (hi, lo).
//
// Streams (128 state rows over the sequence) are dealt to the CTAs in equal shares of chunks, so a stream may be cut
// once and handed on through global memory: 160 streams of 128 chunks took 731 us with whole streams (two waves on
// 148 SMs), 440 in shares.
//
// What bounds it: the chain of a chunk, S -> R -> u -> S, three products and three passes of the T warps over
// their results, about 5400 cycles (3.2 us) per chunk and CTA, of which the 72 products take about 1950 to issue. 24 heads of
// 64 x 128, 8 x 2048 tokens (96 CTAs, 32 chunks each): 104 us; 80 heads, 4 x 8192 (148 CTAs): 440 us. The
// same chain on mma.sync, the state in registers, took 2200 us of the latter and the prep.
//
// kStore is the backward pass's recomputation: no Y, but the state entering each chunk, err and u, rounded to bf16:
// they meet operands that are bf16 already (K, Q, dY) in gradients that are stored in bf16 (relative errors of
// 3.2e-3 against 1.7e-3 for the storage alone); fp32 would double the pass's largest traffic. kParts, for short
// sequences (see in_parts in ssd_delta_mma.cu), leaves err in two bf16 parts alone.
//
// Every wait is bounded (tc_ptx.cuh); one that runs out sets bit 0 of the workspace's status word.
#include "delta_tc.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kTWarps = 16, kOWarp = 4 + kTWarps, kThreads = 32 * (kOWarp + 4);
constexpr int kTriLbo = 128, kTriSbo = 256;  // see tri_rows
constexpr int kTri = 10 * 512;     // bytes of a 64 x 64 lower triangle of 16 x 16 blocks, bf16
constexpr int kTmS = 0, kTmHi = 128, kTmLo = 192, kTmR = 256, kTmY = 320, kTmA = 384, kTmAl = 416;
constexpr int kEk = kTmLo, kEkl = kTmLo + 32;  // ek u over S lo

template <int NT, bool PAIR, bool kStore>
struct Lay {
    static constexpr int HB = PAIR ? 2 : 1;
    static constexpr int k = 0, kBytes = NT / 64 * kPanel;
    static constexpr int q = k + kBytes, x = q + (kStore ? 0 : kBytes), w = x + 2 * kPanel;
    // per head W hi, W lo, P (not kStore), then the scalars
    static constexpr int p = 2 * kTri, scal = p + (kStore ? 0 : kTri), head = scal + 3 * kC * 4;
    static constexpr int stage = (w + HB * head + 1023) / 1024 * 1024;
    static constexpr int out = 2 * stage;                     // O warps' staging, 4 KB each (kStore: u, err and the state)
    static constexpr int bar = out + (kStore ? 2 : 1) * 4 * 4096 + (kStore ? 4 * 64 * NT : 0);
    static constexpr int bytes = bar + 256;
    // what the loader's barrier counts per chunk
    static constexpr int tx = kBytes + (kStore ? 0 : kBytes) + 2 * kPanel + HB * head;
};

struct ChainArgs {
    const float *h0;
    const char *prep;
    int64_t prep_bytes;  // per chunk and head
    int scal_at, rows_at;  // reverse chain: the scalars; W and P by rows of blocks (hi, lo each)
    int nc, H, P, G, N;
    int tiles, streams;  // of 128 rows per head; (tiles x heads or head pairs x batch)
    float *h_final;
    float *hand;  // [CTA][128 rows][NT]: states handed on to the next CTA
    int *flags;   // [CTA]: T warps that have written theirs
    int *status;
    int wait_us;
};

// The chunks of all streams, in order, are cut into equal contiguous shares, one per CTA. A share may
// begin and end inside a stream; its last, begun stream runs first and its first, begun by the CTA
// before, runs last, so that a state handed on is ready long before it is read. Shares are no shorter
// than a stream, so a stream is cut at most once.
struct Seg {
    int stream, c0, c1;
};
struct Share {
    int64_t lo, hi;
    int nc, head, full0, full, n;
    __device__ __forceinline__ Share(int64_t total, int nc_, int i, int grid) : nc(nc_) {
        lo = total * i / grid, hi = total * (i + 1) / grid;
        head = (int)(hi % nc);
        full0 = (int)((lo + nc - 1) / nc);
        full = (int)(hi / nc) - full0;
        n = (head ? 1 : 0) + full + (lo % nc ? 1 : 0);
    }
    __device__ __forceinline__ Seg at(int j) const {
        if (head && j == 0) return Seg{full0 + full, 0, head};
        j -= head ? 1 : 0;
        return j < full ? Seg{full0 + j, 0, nc} : Seg{full0 - 1, (int)(lo % nc), nc};
    }
};

// Bounded wait for `want` arrivals on a counter in global memory.
__device__ __noinline__ bool wait_count(const int *flag, int want, volatile int *abort_flag, int *status) {
    const unsigned long long t0 = now_ns(), lim = wait_limit_ns(abort_flag);
    for (;;) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v >= want) return true;
        if (*abort_flag) return false;
        if (now_ns() - t0 > lim) {
            *abort_flag = 1;
            atomicOr(status, 1);
            return false;
        }
        __nanosleep(200);
    }
}

// State rows as they enter a segment, SC columns from n0 on: handed on by CTA `from`, or the initial state.
template <int SC>
__device__ __forceinline__ void load_rows(uint32_t (&s)[SC], const ChainArgs &a, int from, int p, int64_t srow, int n0, int row, int nt) {
#pragma unroll
    for (int i = 0; i < SC; i += 4) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from >= 0)
            f = __ldcg(reinterpret_cast<const float4 *>(a.hand + ((int64_t)from * 128 + row) * nt + n0 + i));
        else if (a.h0 && p < a.P && n0 + i < a.N)
            f = *reinterpret_cast<const float4 *>(a.h0 + srow * a.N + n0 + i);
        s[i] = __float_as_uint(f.x), s[i + 1] = __float_as_uint(f.y);
        s[i + 2] = __float_as_uint(f.z), s[i + 3] = __float_as_uint(f.w);
    }
}
// And as they leave it: for the CTA that goes on, or the final state.
template <int SC>
__device__ __forceinline__ void store_rows(uint32_t taddr, const ChainArgs &a, bool hand_on, int cta, int p, int64_t srow, int n0,
                                           int row, int nt) {
    float *dst = hand_on ? a.hand + ((int64_t)cta * 128 + row) * nt : a.h_final && p < a.P ? a.h_final + srow * a.N : nullptr;
    const int cols = hand_on ? nt : a.N;
#pragma unroll
    for (int j = 0; j < SC; j += 16) {
        uint32_t s[16];
        tmem_ld16(taddr + n0 + j, s);
        tmem_wait_ld();
        if (dst)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + j + 4 * i < cols)
                    *reinterpret_cast<uint4 *>(dst + n0 + j + 4 * i) = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    }
}
// 32 rows of a bf16 state in TMEM to panels of 64 columns, [32 rows][128 B], swizzled.
template <int NT>
__device__ __forceinline__ void put_state(uint32_t taddr, unsigned char *stage, int lane) {
#pragma unroll
    for (int pn = 0; pn < NT / 64; ++pn) {
        uint32_t v[32];
        tmem_ld32(taddr + 32 * pn, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(stage + pn * 4096 + swz(lane, i)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}
// Pairs of tokens of one row per lane to [64 tokens][32 rows].
__device__ __forceinline__ void put_pairs(const uint32_t (&o)[32], unsigned char *stage, int lane) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        *reinterpret_cast<uint16_t *>(stage + (2 * i) * 64 + 2 * lane) = (uint16_t)(o[i] & 0xffffu);
        *reinterpret_cast<uint16_t *>(stage + (2 * i + 1) * 64 + 2 * lane) = (uint16_t)(o[i] >> 16);
    }
}

template <int NT, bool PAIR, bool kStore, bool kParts>
__device__ __forceinline__ void chain_fwd(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const CUtensorMap &tm_x,
                                          const CUtensorMap &tm_o0, const CUtensorMap &tm_o1, const CUtensorMap &tm_s,
                                          const ChainArgs &a, int cta, int ctas) {
    using Z = Lay<NT, PAIR, kStore>;
    constexpr int HB = Z::HB;
    extern __shared__ __align__(1024) unsigned char sm[];
    if ((smem_u32(sm) & 1023u) != 0) {  // the swizzled layouts need 1024-byte alignment
        if (threadIdx.x == 0) atomicOr(a.status, 2);
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Z::bar);
    uint64_t *full = bar;        // [2] K, Q, x and the scalars of the stage landed
    uint64_t *sfree = bar + 4;   // [2] the stage's readers are done
    uint64_t *rdyR = bar + 6, *rdyE = bar + 7, *rdyS = bar + 8, *rdyQ = bar + 9, *rdyY = bar + 10;  // products done
    uint64_t *sb = bar + 11;     // the state's operands written (T)
    uint64_t *ab = bar + 12;     // beta R written (T)
    uint64_t *ub = bar + 13;     // ek u written (T)
    uint64_t *ost = bar + 3;     // kStore: S hi read (O)
    uint64_t *yu = bar + 2;      // u (kStore: u and err, to go out) written (T)
    uint64_t *ys = bar + 14;     // Yq scaled (O)
    uint64_t *ofree = bar + 15;  // Y (kStore: err and u) read (O)
    uint64_t *fin = bar + 16;
    int *status = a.status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nc = a.nc;
    const Share share((int64_t)a.streams * nc, nc, cta, ctas);
    const int steps = (int)(share.hi - share.lo);
    // batch row, first head and first state row of a stream
    const auto place = [&](int stream, int &b, int &h, int &pc) {
        const int tile = stream % a.tiles, hy = stream / a.tiles % (a.H / HB);
        b = stream / a.tiles / (a.H / HB), h = hy * HB, pc = 128 * tile;
    };

    constexpr int kReaders = 1 + kTWarps + (kStore ? 0 : 4);  // of a stage: the products, T, O
    // in the order above: full, yu, ost, sfree, the five products, sb, ab, ub, ys, ofree, fin
    constexpr int counts[17] = {1, 1, kTWarps, 4, kReaders, kReaders, 1, 1, 1, 1, 1, kTWarps, kTWarps, kTWarps, 4, 4, 1};
    const Setup su = set_up(bar, counts, a.wait_us, warp);
    const uint32_t tmem = su.tmem;
    volatile int *abort_flag = su.abort_flag;
    const auto scal_of = [&](int k, int e) { return reinterpret_cast<const float *>(sm + k * Z::stage + Z::w + e * Z::head + Z::scal); };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
            int it = 0;
            bool ok = true;
            for (int j = 0; ok && j < share.n; ++j) {
                const Seg sg = share.at(j);
                int b, h, pc;
                place(sg.stream, b, h, pc);
                const int grp = h / (a.H / a.G);
                for (int c = sg.c0; c < sg.c1; ++c, ++it) {
                    const int k = it & 1;
                    if (it >= 2 && !(ok = wait_phase(&sfree[k], (uint32_t)((it - 2) >> 1) & 1u, abort_flag, status))) break;
                    unsigned char *st = sm + k * Z::stage;
                    mbar_arrive_tx(&full[k], Z::tx);
                    for (int pn = 0; pn < NT / 64; ++pn)
                        tma_load_4d_hint(st + Z::k + pn * kPanel, &tm_k, &full[k], 64 * pn, grp, c * kC, b, keep);
                    for (int pn = 0; pn < 2; ++pn)
                        tma_load_4d_hint(st + Z::x + pn * kPanel, &tm_x, &full[k], PAIR ? 0 : pc + 64 * pn, PAIR ? h + pn : h, c * kC,
                                         b, stream);
                    for (int e = 0; e < HB; ++e)
                        bulk_load(st + Z::w + e * Z::head, a.prep + (((int64_t)b * a.H + h + e) * nc + c) * a.prep_bytes, Z::head,
                                  &full[k]);
                    if constexpr (!kStore)
                        for (int pn = 0; pn < NT / 64; ++pn)
                            tma_load_4d_hint(st + Z::q + pn * kPanel, &tm_q, &full[k], 64 * pn, grp, c * kC, b, keep);
                }
            }
            drain_loads(full, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        constexpr uint32_t id_ks = idesc(128, 64, false, false), id_s = idesc(128, NT, false, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // A lower triangle as right operand, a column of blocks (16 tokens) at a time, rows from its own block
        // on. No swizzle: core matrices of 128 bytes, the two of a block's row 128 apart, rows of them 256.
        const uint32_t el = elect_one();
        const auto tri = [&](int head, uint32_t d, uint32_t left, uint32_t tile, auto acc) {
            const uint64_t td = (uint64_t)((tile >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(256 >> 4) << 32 |
                                (uint64_t)1 << 46;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t ti = td + (uint64_t)((i * 4 - i * (i - 1) / 2) * 512 >> 4);
                constexpr auto id = [](int i) { return idesc(128, 64 - 16 * i, false, false); };
                if constexpr (PAIR) {
                    if (i == 0)
                        mma_half_el<decltype(acc)::value>(el, head, d, left, ti, id(0));
                    else
                        mma_half_el<true>(el, head, d + 16 * i, left + 8 * i, ti, id(i));
                } else {
                    if (i == 0)
                        mma_el<decltype(acc)::value>(el, d, left, ti, id(0));
                    else
                        mma_el<true>(el, d + 16 * i, left + 8 * i, ti, id(i));
                }
            }
        };
        constexpr std::true_type add{};
        constexpr std::false_type set{};
        for (int c = 0; c < steps; ++c) {
            const int k = c & 1;
            const uint32_t par = (uint32_t)c & 1u;
            const uint32_t st = smem_u32(sm) + k * Z::stage;
            if (!wait_warp(&full[k], (uint32_t)(c >> 1) & 1u, abort_flag, status)) break;
            if (!wait_warp(sb, par, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t kd = sdesc(st + Z::k, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < NT / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4);
                if (kk == 0)
                    mma_el<false>(el, tm + kTmR, tm + kTmLo, kd, id_ks);
                else
                    mma_el<true>(el, tm + kTmR, tm + kTmLo + 8 * kk, kd + off, id_ks);
                mma_el<true>(el, tm + kTmR, tm + kTmHi + 8 * kk, kd + off, id_ks);
            }
            commit_el(el, rdyR);
            if constexpr (!kStore) {
                if (c > 0 && !wait_warp(ofree, par ^ 1u, abort_flag, status)) break;
                tc_fence_after();
                const uint64_t qd = sdesc(st + Z::q, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < NT / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4);
                    if (kk == 0)
                        mma_el<false>(el, tm + kTmY, tm + kTmHi, qd, id_ks);
                    else
                        mma_el<true>(el, tm + kTmY, tm + kTmHi + 8 * kk, qd + off, id_ks);
                }
                commit_el(el, rdyQ);
            }
            if (!wait_warp(ab, par, abort_flag, status)) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < HB; ++e) {
                const uint32_t wh = st + Z::w + e * Z::head;
                tri(e, tm + kTmR, tm + kTmAl, wh, set);
                tri(e, tm + kTmR, tm + kTmA, wh + kTri, add);
                tri(e, tm + kTmR, tm + kTmA, wh, add);
            }
            commit_el(el, rdyE);
            if (!wait_warp(ub, par, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t ks = sdesc(st + Z::k, kPanel, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_el<true>(el, tm + kTmS, tm + kEkl + 8 * kk, ks + 128 * kk, id_s);
                mma_el<true>(el, tm + kTmS, tm + kEk + 8 * kk, ks + 128 * kk, id_s);
            }
            commit_el(el, rdyS);
            if constexpr (!kStore) {
                if (!wait_warp(ys, par, abort_flag, status)) break;
                if (!wait_warp(yu, par, abort_flag, status)) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < HB; ++e) {
                    tri(e, tm + kTmY, tm + kTmAl, st + Z::w + e * Z::head + Z::p, add);
                    tri(e, tm + kTmY, tm + kTmA, st + Z::w + e * Z::head + Z::p, add);
                }
                commit_el(el, rdyY);
            }
            commit_el(el, &sfree[k]);
        }
        commit_el(el, fin);
    } else if (warp < 4) {
        // (idle: a T or O warp's TMEM lanes are those of its number modulo 4)
    } else if (warp < kOWarp) {
        // ------------------------------------------------------------- T: the chain's elementwise links
        const int qtr = warp & 3, sub = (warp - 4) >> 2, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);  // this warp's lanes
        const int pp = (qtr & 1) * 32 + lane;                      // row within the x panel qtr >> 1
        constexpr int SC = NT / 4;  // state columns of this warp, from n0 on
        const int n0 = sub * SC, tk0 = 16 * sub;  // and tokens
        int it = 0;
        bool ok = true;
        for (int j = 0; ok && j < share.n; ++j) {
            const Seg sg = share.at(j);
            int b, h, pc;
            place(sg.stream, b, h, pc);
            const int p = PAIR ? pp : pc + 32 * qtr + lane;  // state row of the head
            const int64_t srow = ((int64_t)b * a.H + h + e) * a.P + p;
            if (sg.c0 > 0 && !(ok = __all_sync(0xffffffffu, wait_count(a.flags + cta - 1, kTWarps, abort_flag, status)))) break;
            int c = sg.c0;
            for (; c < sg.c1; ++c, ++it) {
                const int k = it & 1;
                const uint32_t par = (uint32_t)it & 1u;
                if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
                const float *eg = scal_of(k, e), *ek = eg + kC, *bt = eg + 2 * kC;
                if (it > 0) {
                    if (!wait_warp(rdyS, par ^ 1u, abort_flag, status)) break;
                    if (kStore && !kParts && !wait_warp(ost, par ^ 1u, abort_flag, status)) break;
                    tc_fence_after();
                }
                // The state's operands; then, while S K^T runs, the state times exp(cum_end) for the next product to
                // add to, and what beta R = beta X - beta eg S K^T needs. This warp: tokens tk0 .. + 15.
                float bx[16], be[16];
                const unsigned char *xt = sm + k * Z::stage + Z::x + (qtr >> 1) * kPanel;
                const auto x_at = [&](int i) {
                    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(xt + swz(tk0 + i, pp >> 3) + 2 * (pp & 7)));
                };
                {
                    uint32_t s[SC];
                    if (c > sg.c0) {
                        if constexpr (SC == 32) {
                            tmem_ld32(lo_ + kTmS + n0, s);
                            tmem_wait_ld(s);
                        } else {
                            tmem_ld16(lo_ + kTmS + n0, s);
                            tmem_wait_ld();
                        }
                    } else {
                        load_rows<SC>(s, a, c > 0 ? cta - 1 : -1, p, srow, n0, 32 * qtr + lane, NT);
                    }
#pragma unroll
                    for (int j = 0; j < SC; j += 16) {
                        uint32_t hi[8], lw[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            split2(__uint_as_float(s[j + 2 * i]), __uint_as_float(s[j + 2 * i + 1]), hi[i], lw[i]);
                        tmem_st8(lo_ + kTmHi + (n0 + j) / 2, hi);
                        tmem_st8(lo_ + kTmLo + (n0 + j) / 2, lw);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb);
                    const float gamma = eg[kC - 1];
#pragma unroll
                    for (int j = 0; j < SC; j += 16) {
                        uint32_t v[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 g = mul2(make_float2(gamma, gamma), pair_of(s[j + 2 * i], s[j + 2 * i + 1]));
                            v[2 * i] = __float_as_uint(g.x), v[2 * i + 1] = __float_as_uint(g.y);
                        }
                        tmem_st16(lo_ + kTmS + n0 + j, v);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 g4 = *reinterpret_cast<const float4 *>(eg + tk0 + i), b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                    be[i] = -b4.x * g4.x, be[i + 1] = -b4.y * g4.y, be[i + 2] = -b4.z * g4.z, be[i + 3] = -b4.w * g4.w;
                    bx[i] = b4.x * x_at(i), bx[i + 1] = b4.y * x_at(i + 1), bx[i + 2] = b4.z * x_at(i + 2), bx[i + 3] = b4.w * x_at(i + 3);
                }
                if (!wait_warp(rdyR, par, abort_flag, status)) break;
                tc_fence_after();
                float R[16];
                {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16(lo_ + kTmR + tk0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 br = fma2(make_float2(be[2 * i], be[2 * i + 1]), pair_of(r[2 * i], r[2 * i + 1]),
                                               make_float2(bx[2 * i], bx[2 * i + 1]));
                        split2(br.x, br.y, hi[i], lw[i]);
                    }
                    tmem_st8(lo_ + kTmA + 8 * sub, hi);
                    tmem_st8(lo_ + kTmAl + 8 * sub, lw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ab);
                    // while W (beta R) runs: R itself, and ek beta
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 g4 = *reinterpret_cast<const float4 *>(eg + tk0 + i), b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                        const float4 k4 = *reinterpret_cast<const float4 *>(ek + tk0 + i);
                        R[i] = fmaf(-g4.x, __uint_as_float(r[i]), x_at(i)), R[i + 1] = fmaf(-g4.y, __uint_as_float(r[i + 1]), x_at(i + 1));
                        R[i + 2] = fmaf(-g4.z, __uint_as_float(r[i + 2]), x_at(i + 2));
                        R[i + 3] = fmaf(-g4.w, __uint_as_float(r[i + 3]), x_at(i + 3));
                        be[i] = k4.x * b4.x, be[i + 1] = k4.y * b4.y, be[i + 2] = k4.z * b4.z, be[i + 3] = k4.w * b4.w;
                    }
                }
                // err = R + E, u = beta err; ek u first, which the state waits for
                if (!wait_warp(rdyE, par, abort_flag, status)) break;
                tc_fence_after();
                {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16(lo_ + kTmR + tk0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        R[2 * i] += __uint_as_float(r[2 * i]), R[2 * i + 1] += __uint_as_float(r[2 * i + 1]);
                        const float2 eu = mul2(make_float2(be[2 * i], be[2 * i + 1]), make_float2(R[2 * i], R[2 * i + 1]));
                        split2(eu.x, eu.y, hi[i], lw[i]);
                    }
                    tmem_st8(lo_ + kEk + 8 * sub, hi);
                    tmem_st8(lo_ + kEkl + 8 * sub, lw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ub);
                    if constexpr (kStore) {  // the last chunk's u and err have left
                        if (it > 0 && !wait_warp(ofree, par ^ 1u, abort_flag, status)) break;
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                        const float u[4] = {b4.x * R[i], b4.y * R[i + 1], b4.z * R[i + 2], b4.w * R[i + 3]};
                        if constexpr (kParts) {
                            split2(R[i], R[i + 1], hi[i / 2], lw[i / 2]);
                            split2(R[i + 2], R[i + 3], hi[i / 2 + 1], lw[i / 2 + 1]);
                        } else if constexpr (kStore) {  // u and err go out rounded; no product here takes u itself
                            hi[i / 2] = pack_bf16(u[0], u[1]), hi[i / 2 + 1] = pack_bf16(u[2], u[3]);
                            lw[i / 2] = pack_bf16(R[i], R[i + 1]), lw[i / 2 + 1] = pack_bf16(R[i + 2], R[i + 3]);
                        } else {
                            split2(u[0], u[1], hi[i / 2], lw[i / 2]);
                            split2(u[2], u[3], hi[i / 2 + 1], lw[i / 2 + 1]);
                        }
                    }
                    if constexpr (kStore) {
                        tmem_st8(lo_ + kTmY + 8 * sub, hi);
                        tmem_st8(lo_ + kTmY + 32 + 8 * sub, lw);
                    } else {
                        tmem_st8(lo_ + kTmA + 8 * sub, hi);
                        tmem_st8(lo_ + kTmAl + 8 * sub, lw);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(yu);
                        mbar_arrive(&sfree[k]);
                    }
                }
            }
            // the segment's end: the final state, or the state for the CTA that goes on
            if (c < sg.c1 || !wait_warp(rdyS, (uint32_t)(it - 1) & 1u, abort_flag, status)) break;
            tc_fence_after();
            store_rows<SC>(lo_ + kTmS, a, sg.c1 < nc, cta, p, srow, n0, 32 * qtr + lane, NT);
            if (sg.c1 < nc) {
                __threadfence();
                __syncwarp();
                if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.flags + cta) : "memory");
            }
        }
    } else {
        // ------------------------------------------------------------- O: outputs, 32 state rows x 64 tokens per warp
        const int qtr = warp & 3, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);
        unsigned char *stage0 = sm + Z::out + qtr * 4096, *stage1 = stage0 + 4 * 4096;  // [64 tokens][32 rows]
        unsigned char *stage2 = sm + Z::out + 8 * 4096 + qtr * 64 * NT;  // kStore: [columns / 64][32 rows][128 B], swizzled
        const uint64_t pol = policy_evict_first();
        int it = 0;
        bool ok = true;
        for (int j = 0; ok && j < share.n; ++j) {
            const Seg sg = share.at(j);
            int b, h, pc;
            place(sg.stream, b, h, pc);
            const int p0 = PAIR ? (qtr & 1) * 32 : pc + 32 * qtr;  // first state row of the head
            int c = sg.c0;
            for (; c < sg.c1; ++c, ++it) {
                const int k = it & 1;
                const uint32_t par = (uint32_t)it & 1u;
                if constexpr (!kStore) {
                    if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
                    if (!wait_warp(rdyQ, par, abort_flag, status)) break;
                    tc_fence_after();
                    const float *eg = scal_of(k, e);
#pragma unroll
                    for (int j = 0; j < 64; j += 16) {
                        uint32_t r[16];
                        tmem_ld16(lo_ + kTmY + j, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 g4 = *reinterpret_cast<const float4 *>(eg + j + i);
                            r[i] = __float_as_uint(g4.x * __uint_as_float(r[i])), r[i + 1] = __float_as_uint(g4.y * __uint_as_float(r[i + 1]));
                            r[i + 2] = __float_as_uint(g4.z * __uint_as_float(r[i + 2]));
                            r[i + 3] = __float_as_uint(g4.w * __uint_as_float(r[i + 3]));
                        }
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
                    if constexpr (!kParts) {  // the entering state, as S hi holds it
                        if (!wait_warp(sb, par, abort_flag, status)) break;
                        tc_fence_after();
                        if (lane == 0) bulk_wait_read();  // the staging's last store has read it
                        __syncwarp();
                        put_state<NT>(lo_ + kTmHi, stage2, lane);
                        tc_fence_before();
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ost);
                        if (lane == 0 && p0 < a.P) {
                            const int unit = (b * a.H + h + e) * nc + c;
                            for (int pn = 0; pn < NT / 64; ++pn)
                                if (64 * pn < a.N) tma_store_4d(&tm_s, stage2 + pn * 4096, 64 * pn, p0, unit, 0, pol);
                            bulk_commit();
                        }
                    }
                    if (!wait_warp(yu, par, abort_flag, status)) break;
                }
                tc_fence_after();
                if (lane == 0) bulk_wait_read();
                __syncwarp();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t o[32];
                    tmem_ld32(lo_ + kTmY + 32 * half, o);
                    tmem_wait_ld(o);
                    if (half) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ofree);
                    }
                    if constexpr (kStore) {  // pairs of tokens: u, then err; or err's parts
                        put_pairs(o, half ? stage1 : stage0, lane);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            reinterpret_cast<__nv_bfloat16 *>(stage0 + (32 * half + i) * 64)[lane] = __float2bfloat16_rn(__uint_as_float(o[i]));
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
            ok = c == sg.c1;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tear_down(tmem, fin, warp, lane);
}

// ---------------------------------------------------------------------------------------------
// The chain in reverse, for the backward pass. With D the cotangent of the state leaving a chunk,
//   per chunk                left                      right                               into
//   Z  = P^T dY              dY (shared memory)        P hi, lo  (rows = the sum's tokens)  Z   64 columns
//   F0 = D K^T               D hi, lo (TMEM)           K                                   R   64
//   E  = W^T (beta F)        beta F hi, lo (TMEM)      W hi, lo                            R   (over F0)
//   D += (eg dY)^T Q         eg dY hi, lo (sh. mem.)   Q, columns contiguous               D   N, fp32
//   D -= (eg r)^T K          -eg r hi, lo (TMEM)       K                                   D
// with F = Z + ek F0, z = F + E, r = beta z = dX. Rows, tokens and warps as above, plus warps 2-3, which
// form eg dY. In a PAIR the products with P and W write one head's lanes at a time, as above.
// z and dX go out in bf16, and D hi of every chunk (an operand of k_delta_grads_tc). Both chains share a launch, since
// neither needs the other: 24 heads of 64 x 128, 4 x 2048 tokens, 117 us for both. 768 threads leave
// 80 registers each, and the T warps of both spill (N = 128: 196 bytes in a PAIR, 252 without; 12 to 32 in the forward chain).
template <int NT, bool PAIR>
struct RevLay {
    static constexpr int HB = PAIR ? 2 : 1;
    static constexpr int kBytes = NT / 64 * kPanel;
    static constexpr int k = 0, q = k + 2 * kBytes;                // two stages each
    static constexpr int dy0 = q + 2 * kBytes, dy1 = dy0 + 2 * kPanel;
    static constexpr int e = dy1 + 2 * kPanel;                     // eg dY: hi, lo, two panels each
    static constexpr int out = e + 4 * kPanel;                     // O warps: two buffers of 4 KB each
    static constexpr int w = out + 4 * 8192, p = w + HB * 2 * kTri;  // W hi, lo per head; P hi, lo per head
    static constexpr int scal = p + HB * 2 * kTri;                 // two stages
    static constexpr int bar = scal + 2 * HB * 3 * kC * 4;
    static constexpr int bytes = bar + 256;
    static constexpr int tx = 2 * kBytes + 2 * kPanel + HB * 3 * kC * 4;
};

// Lower triangle by rows of blocks, as right operand whose sum runs over its rows: core matrices of 8 rows by
// 8 columns, the next 8 columns 256 bytes on, the next 8 rows 128.
__device__ __forceinline__ uint64_t tri_rows(uint32_t tile, int a) {
    return (uint64_t)(((tile + 512 * (a * (a + 1) / 2)) >> 4) & 0x3FFFu) | (uint64_t)(kTriLbo >> 4) << 16 |
           (uint64_t)(kTriSbo >> 4) << 32 | (uint64_t)1 << 46;
}
template <int NT, bool PAIR, bool kParts>
__device__ __forceinline__ void chain_rev(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const CUtensorMap &tm_dy,
                                          const CUtensorMap &tm_z, const CUtensorMap &tm_dx, const CUtensorMap &tm_d,
                                          const ChainArgs &a, int cta, int ctas) {
    using Z = RevLay<NT, PAIR>;
    constexpr int HB = Z::HB;
    extern __shared__ __align__(1024) unsigned char sm[];
    if ((smem_u32(sm) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(a.status, 2);
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Z::bar);
    uint64_t *full = bar, *sfree = bar + 2;                    // [2] a stage's loads landed; its readers done
    uint64_t *wfull = bar + 4, *wfree = bar + 5;               // W landed; read
    uint64_t *pfull = bar + 6, *pfree = bar + 7;               // P landed; read
    uint64_t *rdyZ = bar + 8, *rdyR = bar + 9, *rdyE = bar + 10, *rdyS = bar + 11;  // products done
    uint64_t *sb = bar + 12, *ab = bar + 13, *ub = bar + 14, *yu = bar + 15;        // T: D's operands, beta F, eg r; z and dX
    uint64_t *eb = bar + 16;                                   // eg dY written
    uint64_t *ost = bar + 17, *ofree = bar + 18;               // O: D hi read; z and dX read
    uint64_t *fin = bar + 19;
    int *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nc = a.nc;
    const Share share((int64_t)a.streams * nc, nc, cta, ctas);
    const int steps = (int)(share.hi - share.lo);
    const auto place = [&](int stream, int &b, int &h, int &pc) {
        const int tile = stream % a.tiles, hy = stream / a.tiles % (a.H / HB);
        b = stream / a.tiles / (a.H / HB), h = hy * HB, pc = 128 * tile;
    };
    constexpr int counts[20] = {1, 1, 1 + kTWarps, 1 + kTWarps, 1, 1, 1, 1, 1, 1, 1, 1, kTWarps, kTWarps, kTWarps, kTWarps, 2, 4, 4, 1};
    const Setup su = set_up(bar, counts, a.wait_us, warp);
    const uint32_t tmem = su.tmem;
    volatile int *abort_flag = su.abort_flag;
    const auto scal_of = [&](int k, int e) { return reinterpret_cast<const float *>(sm + Z::scal + (k * HB + e) * 3 * kC * 4); };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
            int it = 0, pp = 0, wp = 0;  // uses of the stages; of P; of W
            bool ok = true;
            for (int j = 0; ok && j < share.n; ++j) {
                const Seg sg = share.at(j);
                int b, h, pc;
                place(sg.stream, b, h, pc);
                const int grp = h / (a.H / a.G);
                for (int t = sg.c0; t < sg.c1; ++t) {
                    const int c = nc - 1 - t, k = it & 1;
                    const auto prep = [&](int e) { return a.prep + (((int64_t)b * a.H + h + e) * nc + c) * a.prep_bytes; };
                    if (it >= 2 && !(ok = wait_phase(&sfree[k], (uint32_t)((it - 2) >> 1) & 1u, abort_flag, status))) break;
                    mbar_arrive_tx(&full[k], Z::tx);
                    for (int pn = 0; pn < 2; ++pn)
                        tma_load_4d_hint(sm + (pn ? Z::dy1 : Z::dy0) + k * kPanel, &tm_dy, &full[k], PAIR ? 0 : pc + 64 * pn,
                                         PAIR ? h + pn : h, c * kC, b, stream);
                    for (int e = 0; e < HB; ++e)
                        bulk_load(sm + Z::scal + (k * HB + e) * 3 * kC * 4, prep(e) + a.scal_at, 3 * kC * 4, &full[k]);
                    for (int pn = 0; pn < NT / 64; ++pn) {
                        tma_load_4d_hint(sm + Z::k + k * Z::kBytes + pn * kPanel, &tm_k, &full[k], 64 * pn, grp, c * kC, b, keep);
                        tma_load_4d_hint(sm + Z::q + k * Z::kBytes + pn * kPanel, &tm_q, &full[k], 64 * pn, grp, c * kC, b, keep);
                    }
                    ++it;
                    // P as soon as the last chunk's Z is done (its products come first in a chunk), then W
                    if (wp > 0 && !(ok = wait_phase(pfree, (uint32_t)(wp - 1) & 1u, abort_flag, status))) break;
                    mbar_arrive_tx(pfull, HB * 2 * kTri);
                    for (int e = 0; e < HB; ++e)
                        bulk_load(sm + Z::p + e * 2 * kTri, prep(e) + a.rows_at + 2 * kTri, 2 * kTri, pfull);
                    ++pp;
                    if (wp > 0 && !(ok = wait_phase(wfree, (uint32_t)(wp - 1) & 1u, abort_flag, status))) break;
                    mbar_arrive_tx(wfull, HB * 2 * kTri);
                    for (int e = 0; e < HB; ++e) bulk_load(sm + Z::w + e * 2 * kTri, prep(e) + a.rows_at, 2 * kTri, wfull);
                    ++wp;
                }
            }
            drain_loads(full, it);
            if (pp > 0) {
                const unsigned long long w0 = now_ns();
                while (!(mbar_try(pfull, (uint32_t)(pp - 1) & 1u) && (wp == 0 || mbar_try(wfull, (uint32_t)(wp - 1) & 1u))) &&
                       now_ns() - w0 < kWaitNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        constexpr uint32_t id_ks = idesc(128, 64, false, false), id_s = idesc(128, NT, false, true), id_eq = idesc(128, NT, true, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t el = elect_one(), base = smem_u32(sm);
        for (int it = 0; it < steps; ++it) {
            const int k = it & 1;
            const uint32_t par = (uint32_t)it & 1u;
            const uint32_t ka = base + Z::k + k * Z::kBytes, qa = base + Z::q + k * Z::kBytes;
            if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
            if (!wait_warp(pfull, par, abort_flag, status)) break;
            if (it > 0 && !wait_warp(ofree, par ^ 1u, abort_flag, status)) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < HB; ++e) {
                const uint64_t ya = sdesc(base + Z::dy0 + k * kPanel, Z::dy1 - Z::dy0, 1024);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const uint64_t right = tri_rows(base + Z::p + (2 * e + 1 - part) * kTri, i);
                        const uint32_t id = idesc(128, 16 * (i + 1), true, true);
                        if constexpr (PAIR)
                            mma_ss_half_el(el, e, tm + kTmY, ya + 128 * i, right, id, part > 0 || i < 3);
                        else
                            mma_ss_el(el, tm + kTmY, ya + 128 * i, right, id, part > 0 || i < 3);
                    }
            }
            commit_el(el, rdyZ);
            commit_el(el, pfree);
            if (!wait_warp(sb, par, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t kd = sdesc(ka, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < NT / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4);
                if (kk == 0)
                    mma_el<false>(el, tm + kTmR, tm + kTmLo, kd, id_ks);
                else
                    mma_el<true>(el, tm + kTmR, tm + kTmLo + 8 * kk, kd + off, id_ks);
                mma_el<true>(el, tm + kTmR, tm + kTmHi + 8 * kk, kd + off, id_ks);
            }
            commit_el(el, rdyR);
            if (!wait_warp(wfull, par, abort_flag, status)) break;
            if (!wait_warp(ab, par, abort_flag, status)) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < HB; ++e)
#pragma unroll
                for (int part = 0; part < 3; ++part)  // lo W hi, hi W lo, hi W hi
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const uint32_t left = tm + (part == 0 ? kTmAl : kTmA) + 8 * i;
                        const uint64_t right = tri_rows(base + Z::w + (2 * e + (part == 1 ? 1 : 0)) * kTri, i);
                        const uint32_t id = idesc(128, 16 * (i + 1), false, true);
                        if constexpr (PAIR) {
                            if (part == 0 && i == 3)
                                mma_half_el<false>(el, e, tm + kTmR, left, right, id);
                            else
                                mma_half_el<true>(el, e, tm + kTmR, left, right, id);
                        } else {
                            if (part == 0 && i == 3)
                                mma_el<false>(el, tm + kTmR, left, right, id);
                            else
                                mma_el<true>(el, tm + kTmR, left, right, id);
                        }
                    }
            commit_el(el, rdyE);
            commit_el(el, wfree);
            if (!wait_warp(eb, par, abort_flag, status)) break;
            tc_fence_after();
            const uint64_t qs = sdesc(qa, kPanel, 1024), ks = sdesc(ka, kPanel, 1024), ed = sdesc(base + Z::e, kPanel, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_ss_el(el, tm + kTmS, ed + 128 * kk + (uint64_t)(2 * kPanel >> 4), qs + 128 * kk, id_eq, 1);
                mma_ss_el(el, tm + kTmS, ed + 128 * kk, qs + 128 * kk, id_eq, 1);
            }
            if (!wait_warp(ub, par, abort_flag, status)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_el<true>(el, tm + kTmS, tm + kEkl + 8 * kk, ks + 128 * kk, id_s);
                mma_el<true>(el, tm + kTmS, tm + kEk + 8 * kk, ks + 128 * kk, id_s);
            }
            commit_el(el, rdyS);
            commit_el(el, &sfree[k]);
        }
        commit_el(el, fin);
    } else if (warp < 4) {
        // ------------------------------------------------------------- eg dY, hi and lo, 16 bytes of a token at a time
        for (int it = 0; it < steps; ++it) {
            const int k = it & 1;
            if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
            if (it > 0 && !wait_warp(rdyS, ((uint32_t)it & 1u) ^ 1u, abort_flag, status)) break;
            // four vectors are read before the first is written: through one array, the compiler keeps the order
#pragma unroll
            for (int v0 = 0; v0 < 16; v0 += 4) {
                uint4 y[4];
                float g[4];
                uint32_t at[4];
                const int pn = v0 >> 3;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = (v0 & 7) * 64 + v * 64 + (warp & 1) * 32 + lane;
                    at[v] = swz(i >> 3, i & 7);
                    y[v] = *reinterpret_cast<const uint4 *>(sm + (pn ? Z::dy1 : Z::dy0) + k * kPanel + at[v]);
                    g[v] = scal_of(k, PAIR ? pn : 0)[i >> 3];
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t in[4] = {y[v].x, y[v].y, y[v].z, y[v].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 m = mul2(make_float2(g[v], g[v]), make_float2(bf16_lo(in[e]), bf16_hi(in[e])));
                        split2(m.x, m.y, hi[e], lo[e]);
                    }
                    *reinterpret_cast<uint4 *>(sm + Z::e + pn * kPanel + at[v]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(sm + Z::e + (2 + pn) * kPanel + at[v]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(eb);
        }
    } else if (warp < kOWarp) {
        // ------------------------------------------------------------- T
        const int qtr = warp & 3, sub = (warp - 4) >> 2, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);
        constexpr int SC = NT / 4;
        const int n0 = sub * SC, tk0 = 16 * sub;
        int it = 0;
        bool ok = true;
        for (int j = 0; ok && j < share.n; ++j) {
            const Seg sg = share.at(j);
            int b, h, pc;
            place(sg.stream, b, h, pc);
            const int p = PAIR ? (qtr & 1) * 32 + lane : pc + 32 * qtr + lane;
            const int64_t srow = ((int64_t)b * a.H + h + e) * a.P + p;
            if (sg.c0 > 0 && !(ok = __all_sync(0xffffffffu, wait_count(a.flags + cta - 1, kTWarps, abort_flag, status)))) break;
            int t = sg.c0;
            for (; t < sg.c1; ++t, ++it) {
                const int k = it & 1;
                const uint32_t par = (uint32_t)it & 1u;
                if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
                const float *eg = scal_of(k, e), *ek = eg + kC, *bt = eg + 2 * kC;
                if (it > 0) {
                    if (!wait_warp(rdyS, par ^ 1u, abort_flag, status)) break;
                    if (!kParts && !wait_warp(ost, par ^ 1u, abort_flag, status)) break;
                    tc_fence_after();
                }
                {  // D's operands; then D times exp(cum_end)
                    uint32_t s[SC];
                    if (t > sg.c0) {
                        if constexpr (SC == 32) {
                            tmem_ld32(lo_ + kTmS + n0, s);
                            tmem_wait_ld(s);
                        } else {
                            tmem_ld16(lo_ + kTmS + n0, s);
                            tmem_wait_ld();
                        }
                    } else {
                        load_rows<SC>(s, a, t > 0 ? cta - 1 : -1, p, srow, n0, 32 * qtr + lane, NT);
                    }
#pragma unroll
                    for (int i0 = 0; i0 < SC; i0 += 16) {
                        uint32_t hi[8], lw[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            split2(__uint_as_float(s[i0 + 2 * i]), __uint_as_float(s[i0 + 2 * i + 1]), hi[i], lw[i]);
                        tmem_st8(lo_ + kTmHi + (n0 + i0) / 2, hi);
                        tmem_st8(lo_ + kTmLo + (n0 + i0) / 2, lw);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb);
                    const float gamma = eg[kC - 1];
#pragma unroll
                    for (int i0 = 0; i0 < SC; i0 += 16) {
                        uint32_t v[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 g = mul2(make_float2(gamma, gamma), pair_of(s[i0 + 2 * i], s[i0 + 2 * i + 1]));
                            v[2 * i] = __float_as_uint(g.x), v[2 * i + 1] = __float_as_uint(g.y);
                        }
                        tmem_st16(lo_ + kTmS + n0 + i0, v);
                    }
                }
                // beta F = beta Z + beta ek D K^T
                float F[16], be[16];
                if (!wait_warp(rdyZ, par, abort_flag, status)) break;
                tc_fence_after();
                uint32_t zf[16];
                tmem_ld16(lo_ + kTmY + tk0, zf);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(ek + tk0 + i), b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                    be[i] = b4.x * k4.x, be[i + 1] = b4.y * k4.y, be[i + 2] = b4.z * k4.z, be[i + 3] = b4.w * k4.w;
                    F[i] = b4.x * __uint_as_float(zf[i]), F[i + 1] = b4.y * __uint_as_float(zf[i + 1]);
                    F[i + 2] = b4.z * __uint_as_float(zf[i + 2]), F[i + 3] = b4.w * __uint_as_float(zf[i + 3]);
                }
                if (!wait_warp(rdyR, par, abort_flag, status)) break;
                tc_fence_after();
                {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16(lo_ + kTmR + tk0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 bf = fma2(make_float2(be[2 * i], be[2 * i + 1]), pair_of(r[2 * i], r[2 * i + 1]),
                                               make_float2(F[2 * i], F[2 * i + 1]));
                        split2(bf.x, bf.y, hi[i], lw[i]);
                    }
                    tmem_st8(lo_ + kTmA + 8 * sub, hi);
                    tmem_st8(lo_ + kTmAl + 8 * sub, lw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ab);
                    // while W^T (beta F) runs: F itself, and -eg beta
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 g4 = *reinterpret_cast<const float4 *>(eg + tk0 + i), b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                        const float4 k4 = *reinterpret_cast<const float4 *>(ek + tk0 + i);
                        F[i] = fmaf(k4.x, __uint_as_float(r[i]), __uint_as_float(zf[i]));
                        F[i + 1] = fmaf(k4.y, __uint_as_float(r[i + 1]), __uint_as_float(zf[i + 1]));
                        F[i + 2] = fmaf(k4.z, __uint_as_float(r[i + 2]), __uint_as_float(zf[i + 2]));
                        F[i + 3] = fmaf(k4.w, __uint_as_float(r[i + 3]), __uint_as_float(zf[i + 3]));
                        be[i] = -g4.x * b4.x, be[i + 1] = -g4.y * b4.y, be[i + 2] = -g4.z * b4.z, be[i + 3] = -g4.w * b4.w;
                    }
                }
                // z = F + E, r = beta z; -eg r first, which D waits for
                if (!wait_warp(rdyE, par, abort_flag, status)) break;
                tc_fence_after();
                {
                    uint32_t r[16], hi[8], lw[8];
                    tmem_ld16(lo_ + kTmR + tk0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        F[2 * i] += __uint_as_float(r[2 * i]), F[2 * i + 1] += __uint_as_float(r[2 * i + 1]);
                        const float2 er = mul2(make_float2(be[2 * i], be[2 * i + 1]), make_float2(F[2 * i], F[2 * i + 1]));
                        split2(er.x, er.y, hi[i], lw[i]);
                    }
                    tmem_st8(lo_ + kEk + 8 * sub, hi);
                    tmem_st8(lo_ + kEkl + 8 * sub, lw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ub);
                    // z and dX, rounded, or z's parts, over Z (which every T warp has read by now)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        if constexpr (kParts) {
                            split2(F[i], F[i + 1], hi[i / 2], lw[i / 2]);
                            split2(F[i + 2], F[i + 3], hi[i / 2 + 1], lw[i / 2 + 1]);
                            continue;
                        }
                        const float4 b4 = *reinterpret_cast<const float4 *>(bt + tk0 + i);
                        hi[i / 2] = pack_bf16(F[i], F[i + 1]), hi[i / 2 + 1] = pack_bf16(F[i + 2], F[i + 3]);
                        lw[i / 2] = pack_bf16(b4.x * F[i], b4.y * F[i + 1]), lw[i / 2 + 1] = pack_bf16(b4.z * F[i + 2], b4.w * F[i + 3]);
                    }
                    tmem_st8(lo_ + kTmY + 8 * sub, hi);
                    tmem_st8(lo_ + kTmY + 32 + 8 * sub, lw);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(yu);
                        mbar_arrive(&sfree[k]);
                    }
                }
            }
            if (t < sg.c1 || !wait_warp(rdyS, (uint32_t)(it - 1) & 1u, abort_flag, status)) break;
            tc_fence_after();
            store_rows<SC>(lo_ + kTmS, a, sg.c1 < nc, cta, p, srow, n0, 32 * qtr + lane, NT);
            if (sg.c1 < nc) {
                __threadfence();
                __syncwarp();
                if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.flags + cta) : "memory");
            }
        }
    } else {
        // ------------------------------------------------------------- O
        const int qtr = warp & 3, e = PAIR ? qtr >> 1 : 0;
        const uint32_t lo_ = tmem + ((uint32_t)(32 * qtr) << 16);
        unsigned char *stage = sm + Z::out + qtr * 8192;  // D hi: [64 columns][32 rows][128 B]; z, dX: [64 tokens][32 rows]
        const uint64_t pol = policy_evict_first();
        int it = 0;
        bool ok = true;
        for (int j = 0; ok && j < share.n; ++j) {
            const Seg sg = share.at(j);
            int b, h, pc;
            place(sg.stream, b, h, pc);
            const int p0 = PAIR ? (qtr & 1) * 32 : pc + 32 * qtr;
            int t = sg.c0;
            for (; t < sg.c1; ++t, ++it) {
                const int c = nc - 1 - t;
                const uint32_t par = (uint32_t)it & 1u;
                if constexpr (!kParts) {
                    if (!wait_warp(sb, par, abort_flag, status)) break;
                    tc_fence_after();
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                    put_state<NT>(lo_ + kTmHi, stage, lane);
                    tc_fence_before();
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ost);
                    if (lane == 0 && p0 < a.P) {
                        const int unit = (b * a.H + h + e) * nc + c;
                        for (int pn = 0; pn < NT / 64; ++pn)
                            if (64 * pn < a.N) tma_store_4d(&tm_d, stage + pn * 4096, 64 * pn, p0, unit, 0, pol);
                        bulk_commit();
                    }
                }
                if (!wait_warp(yu, par, abort_flag, status)) break;
                tc_fence_after();
                if (lane == 0) bulk_wait_read();
                __syncwarp();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t o[32];
                    tmem_ld32(lo_ + kTmY + 32 * half, o);
                    tmem_wait_ld(o);
                    if (half) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ofree);
                    }
                    put_pairs(o, stage + 4096 * half, lane);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0 && p0 < a.P) {
                    tma_store_4d(&tm_z, stage, p0, h + e, c * kC, b, pol);
                    tma_store_4d(&tm_dx, stage + 4096, p0, h + e, c * kC, b, pol);
                    bulk_commit();
                }
            }
            ok = t == sg.c1;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tear_down(tmem, fin, warp, lane);
}

struct Maps {
    CUtensorMap k, q, x, o0, o1, s;
};

template <int NT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) k_delta_tc(const __grid_constant__ Maps m, const __grid_constant__ ChainArgs a) {
    chain_fwd<NT, PAIR, false, false>(m.k, m.q, m.x, m.o0, m.o1, m.s, a, blockIdx.x, gridDim.x);
}

// Both chains of the backward pass, which do not depend on one another: the first half of the CTAs
// recomputes the states, the other half walks back.
template <int NT, bool PAIR, bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    k_delta_tc_bwd(const __grid_constant__ Maps mf, const __grid_constant__ Maps mr, const __grid_constant__ ChainArgs f,
                   const __grid_constant__ ChainArgs r) {
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half)
        chain_fwd<NT, PAIR, true, kParts>(mf.k, mf.q, mf.x, mf.o0, mf.o1, mf.s, f, blockIdx.x, half);
    else
        chain_rev<NT, PAIR, kParts>(mr.k, mr.q, mr.x, mr.o0, mr.o1, mr.s, r, blockIdx.x - half, half);
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

// [units, P, N] bf16 states, boxes of 64 columns by 32 rows, 128-byte swizzle.
bool encode_states(CUtensorMap *m, const void *base, int64_t N, int64_t P, int64_t units) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)N, (cuuint64_t)P, (cuuint64_t)units, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)(N * 2), (cuuint64_t)(P * N * 2), (cuuint64_t)(units * P * N * 2)};
    const cuuint32_t box[4] = {64, 32, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Two heads of a group side by side where each fits 64 rows: half the streams, and K, Q loaded once for
// both.
bool pairs(const DeltaProblem &p) { return p.P <= 64 && (p.H / p.G) % 2 == 0; }
int64_t streams_of(const DeltaProblem &p) { return pairs(p) ? p.B * (p.H / 2) : p.B * p.H * ((p.P + 127) / 128); }

bool encode_maps(Maps *m, const DeltaProblem &p, const void *x, const void *o0, const void *o1, const void *states) {
    const int64_t units = p.B * p.H * ((p.L + kC - 1) / kC);
    if (!encode_4d(&m->k, p.Bm, p.N, p.G, p.L, p.B, kC) || !encode_4d(&m->q, p.Cm, p.N, p.G, p.L, p.B, kC) ||
        !encode_4d(&m->x, x, p.P, p.H, p.L, p.B, kC) || !encode_out(&m->o0, o0, p.P, p.H, p.L, p.B))
        return false;
    m->o1 = m->o0;
    m->s = m->o0;
    return (!o1 || encode_out(&m->o1, o1, p.P, p.H, p.L, p.B)) && (!states || encode_states(&m->s, states, p.N, p.P, units));
}

template <typename K, typename... A>
cudaError_t launch(K kernel, int grid, int smem, bool cut, cudaStream_t s, const A &...args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    // Where a stream is cut its CTAs have to be resident together, which a cooperative launch guarantees.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cut ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

ChainArgs args_of(const DeltaProblem &p, const DeltaChain &ch, const float *first, float *last, int cta0) {
    const int tiles = pairs(p) ? 1 : (int)((p.P + 127) / 128);
    return ChainArgs{first, ch.prep, ch.prep_bytes, ch.scal_at, ch.rows_at, (int)((p.L + kC - 1) / kC), (int)p.H, (int)p.P,
                     (int)p.G, (int)p.N, tiles, (int)streams_of(p), last, ch.hand + (int64_t)cta0 * 128 * (p.N <= 64 ? 64 : 128),
                     ch.flags + cta0, ch.status, wait_limit_us()};
}

template <int NT, bool PAIR>
cudaError_t fwd(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    Maps m;
    if (!encode_maps(&m, p, p.x, p.y, nullptr, nullptr)) return cudaErrorInvalidValue;
    const int grid = delta_tc_grid(p, false);
    return launch(k_delta_tc<NT, PAIR>, grid, Lay<NT, PAIR, false>::bytes, streams_of(p) > grid, s, m,
                  args_of(p, ch, p.h0, p.h_final, 0));
}

template <int NT, bool PAIR>
cudaError_t bwd(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, cudaStream_t s) {
    Maps mf, mr;
    const bool parts = ch.z_lo;
    if (!(parts ? encode_maps(&mf, p, p.x, ch.err, ch.u, nullptr) && encode_maps(&mr, p, g.dy, ch.z, ch.z_lo, nullptr)
                : encode_maps(&mf, p, p.x, ch.u, ch.err, ch.states) && encode_maps(&mr, p, g.dy, ch.z, g.dx, ch.cots)))
        return cudaErrorInvalidValue;
    const int grid = delta_tc_grid(p, true);
    constexpr int f = Lay<NT, PAIR, true>::bytes, r = RevLay<NT, PAIR>::bytes;
    return launch(parts ? k_delta_tc_bwd<NT, PAIR, true> : k_delta_tc_bwd<NT, PAIR, false>, grid, f > r ? f : r, streams_of(p) > grid / 2,
                  s, mf, mr, args_of(p, ch, p.h0, nullptr, 0), args_of(p, ch, g.dh_final, g.dh0, grid / 2));
}

}  // namespace

// One CTA per SM (it takes all of TMEM), or per stream where there are fewer; half of them for each of
// the backward pass's two chains.
int delta_tc_grid(const DeltaProblem &p, bool backward) {
    const int sms = sm_count(), most = backward ? sms / 2 : sms;
    const int64_t streams = streams_of(p);
    return (int)(streams < most ? streams : most) * (backward ? 2 : 1);
}

size_t delta_tc_hand_bytes(const DeltaProblem &p, bool backward) {
    const int grid = delta_tc_grid(p, backward);
    return streams_of(p) > (backward ? grid / 2 : grid) ? (size_t)grid * 128 * (p.N <= 64 ? 64 : 128) * sizeof(float) : 0;
}

cudaError_t delta_tc_fwd(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    if (p.N <= 64) return pairs(p) ? fwd<64, true>(p, ch, s) : fwd<64, false>(p, ch, s);
    return pairs(p) ? fwd<128, true>(p, ch, s) : fwd<128, false>(p, ch, s);
}

cudaError_t delta_tc_bwd(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, cudaStream_t s) {
    if (p.N <= 64) return pairs(p) ? bwd<64, true>(p, g, ch, s) : bwd<64, false>(p, g, ch, s);
    return pairs(p) ? bwd<128, true>(p, g, ch, s) : bwd<128, false>(p, g, ch, s);
}

}  // namespace ssd
