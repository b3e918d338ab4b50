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
// Warps (768 threads): 0 loads (TMA), 1 issues the products, 4-19 (T) form R, u and the state's operands (four warps per 32 lanes, a quarter of the
// columns each), 20-23 (O) scale Yq and write Y out. TMEM, 512 columns: S 128, S hi 64, S lo 64 (later
// ek u), R 64, Y 64, beta R then u 2 x 64.
//
// What bounds it: the chain of a chunk, S -> R -> u -> S, each link a product (0.1-0.25 us) and a pass of
// the T warps over its result (0.25-0.35 us).
//
// kStore is the backward pass's recomputation: no Y, but the state entering each chunk, err and u in bf16.
//
// Every wait is bounded (tc_ptx.cuh); one that runs out sets bit 0 of the workspace's status word.
#include <type_traits>

#include "ssd_delta.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kC = kDeltaChunk;
constexpr int kTWarps = 16, kOWarp = 4 + kTWarps, kThreads = 32 * (kOWarp + 4);
constexpr int kPanel = kC * 128;   // bytes of 64 rows of 64 bf16
constexpr int kTri = 10 * 512;     // bytes of a 64 x 64 lower triangle of 16 x 16 blocks, bf16
constexpr int kTmS = 0, kTmHi = 128, kTmLo = 192, kTmR = 256, kTmY = 320, kTmA = 384, kTmAl = 448;
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

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The products are issued by one elected thread, but from code that the whole warp runs: descriptors and
// TMEM addresses then stay in uniform registers. From inside `if (lane == 0)` each product took about 90
// cycles to issue, most of them moving its operands into uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r;
}
template <bool kAcc>
__device__ __forceinline__ void mma_el(uint32_t leader, uint32_t d, uint32_t left, uint64_t right, uint32_t id) {
    if constexpr (kAcc)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 p, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(left), "l"(right), "r"(id), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 p, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(left), "l"(right), "r"(id), "r"(leader)
            : "memory");
}
__device__ __forceinline__ void commit_el(uint32_t leader, uint64_t *bar) {
    if (leader) mma_commit(bar);
    __syncwarp();
}

// hi + lo parts of a pair of fp32 values (lo: what hi leaves, rounded: 2^-18 of the value at worst)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    asm("{\n\t.reg .b64 v, h, m;\n\t.reg .f32 a, b;\n\t"
        "mov.b64 v, {%1, %2};\n\tmov.b64 h, {%3, %4};\n\tmov.b64 m, {%5, %5};\n\t"
        "fma.rn.f32x2 v, h, m, v;\n\tmov.b64 {a, b}, v;\n\tcvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(lo)
        : "f"(x), "f"(y), "f"(bf16_lo(hi)), "f"(bf16_hi(hi)), "f"(-1.f));
}
// packed pairs of fp32: a b, and c + a b
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 pair_of(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }

template <int NT, bool PAIR, bool kStore>
__global__ void __launch_bounds__(kThreads, 1)
    k_delta_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_o0,
               const __grid_constant__ CUtensorMap tm_o1, const __grid_constant__ CUtensorMap tm_s, const ChainArgs a) {
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 17);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bar + 18);
    int *status = a.status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nc = a.nc;
    const Share share((int64_t)a.streams * nc, nc, blockIdx.x, gridDim.x);
    const int steps = (int)(share.hi - share.lo);
    // batch row, first head and first state row of a stream
    const auto place = [&](int stream, int &b, int &h, int &pc) {
        const int tile = stream % a.tiles, hy = stream / a.tiles % (a.H / HB);
        b = stream / a.tiles / (a.H / HB), h = hy * HB, pc = 128 * tile;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&sfree[i], 1 + kTWarps + (kStore ? 0 : 4));  // the products, T, O
        }
        mbar_init(rdyR, 1);
        mbar_init(rdyE, 1);
        mbar_init(rdyS, 1);
        mbar_init(rdyQ, 1);
        mbar_init(rdyY, 1);
        mbar_init(sb, kTWarps);
        mbar_init(ab, kTWarps);
        mbar_init(ub, kTWarps);
        mbar_init(yu, kTWarps);
        mbar_init(ys, 4);
        mbar_init(ofree, 4);
        mbar_init(ost, 4);
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
            // loads in flight land before the CTA exits
            for (int i = 1; i <= 2; ++i) {
                if (it - i < 0) continue;
                const unsigned long long w0 = now_ns();
                while (!mbar_try(&full[(it - i) & 1], (uint32_t)((it - i) >> 1) & 1u) && now_ns() - w0 < kWaitNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        constexpr uint32_t id_ks = idesc(128, 64, false, false), id_s = idesc(128, NT, false, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // A lower triangle as right operand, a column of blocks (16 tokens) at a time, rows from its own block
        // on. No swizzle: core matrices of 128 bytes, the two of a block's row 128 apart, rows of them 256.
        const uint32_t el = elect_one();
        const auto tri = [&](uint32_t d, uint32_t left, uint32_t tile, auto acc) {
            const uint64_t td = (uint64_t)((tile >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(256 >> 4) << 32 |
                                (uint64_t)1 << 46;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t ti = td + (uint64_t)((i * 4 - i * (i - 1) / 2) * 512 >> 4);
                if (i == 0)
                    mma_el<decltype(acc)::value>(el, d, left, ti, idesc(128, 64, false, false));
                else
                    mma_el<true>(el, d + 16 * i, left + 8 * i, ti, idesc(128, 64 - 16 * i, false, false));
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
                if (e == 0)
                    tri(tm + kTmR, tm + kTmAl, wh, set);
                else
                    tri(tm + kTmR, tm + kTmAl + 32 * e, wh, add);
                tri(tm + kTmR, tm + kTmA + 32 * e, wh + kTri, add);
                tri(tm + kTmR, tm + kTmA + 32 * e, wh, add);
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
                    tri(tm + kTmY, tm + kTmAl + 32 * e, st + Z::w + e * Z::head + Z::p, add);
                    tri(tm + kTmY, tm + kTmA + 32 * e, st + Z::w + e * Z::head + Z::p, add);
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
        if constexpr (PAIR) {  // zeros in the other head's tokens
            const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            tmem_st8(lo_ + kTmA + 32 * (1 - e) + 8 * sub, zero);
            tmem_st8(lo_ + kTmAl + 32 * (1 - e) + 8 * sub, zero);
        }
        int it = 0;
        bool ok = true;
        for (int j = 0; ok && j < share.n; ++j) {
        const Seg sg = share.at(j);
        int b, h, pc;
        place(sg.stream, b, h, pc);
        const int p = PAIR ? pp : pc + 32 * qtr + lane;  // state row of the head
        const int64_t srow = ((int64_t)b * a.H + h + e) * a.P + p;
        if (sg.c0 > 0 && !(ok = __all_sync(0xffffffffu, wait_count(a.flags + blockIdx.x - 1, kTWarps, abort_flag, status)))) break;
        int c = sg.c0;
        for (; c < sg.c1; ++c, ++it) {
            const int k = it & 1;
            const uint32_t par = (uint32_t)it & 1u;
            if (!wait_warp(&full[k], (uint32_t)(it >> 1) & 1u, abort_flag, status)) break;
            const float *eg = scal_of(k, e), *ek = eg + kC, *bt = eg + 2 * kC;
            if (it > 0) {
                if (!wait_warp(rdyS, par ^ 1u, abort_flag, status)) break;
                if (kStore && !wait_warp(ost, par ^ 1u, abort_flag, status)) break;
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
#pragma unroll
                    for (int i = 0; i < SC; i += 4) {
                        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (c > 0)
                            f = __ldcg(reinterpret_cast<const float4 *>(a.hand + ((int64_t)(blockIdx.x - 1) * 128 + 32 * qtr + lane) * NT + n0 + i));
                        else if (a.h0 && p < a.P && n0 + i < a.N)
                            f = *reinterpret_cast<const float4 *>(a.h0 + srow * a.N + n0 + i);
                        s[i] = __float_as_uint(f.x), s[i + 1] = __float_as_uint(f.y);
                        s[i + 2] = __float_as_uint(f.z), s[i + 3] = __float_as_uint(f.w);
                    }
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
                tmem_st8(lo_ + kTmA + 32 * e + 8 * sub, hi);
                tmem_st8(lo_ + kTmAl + 32 * e + 8 * sub, lw);
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
                    if constexpr (kStore) {  // u and err go out rounded; no product here takes u itself
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
                    tmem_st8(lo_ + kTmA + 32 * e + 8 * sub, hi);
                    tmem_st8(lo_ + kTmAl + 32 * e + 8 * sub, lw);
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
        float *dst = sg.c1 < nc ? a.hand + ((int64_t)blockIdx.x * 128 + 32 * qtr + lane) * NT
                                : a.h_final && p < a.P ? a.h_final + srow * a.N : nullptr;
        const int cols = sg.c1 < nc ? NT : a.N;
#pragma unroll
        for (int jj = 0; jj < SC; jj += 16) {
            uint32_t s[16];
            tmem_ld16(lo_ + kTmS + n0 + jj, s);
            tmem_wait_ld();
            if (dst)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + jj + 4 * i < cols)
                        *reinterpret_cast<uint4 *>(dst + n0 + jj + 4 * i) = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
        }
        if (sg.c1 < nc) {
            __threadfence();
            __syncwarp();
            if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.flags + blockIdx.x) : "memory");
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
            } else {  // the entering state, as S hi holds it
                if (!wait_warp(sb, par, abort_flag, status)) break;
                tc_fence_after();
                if (lane == 0) bulk_wait_read();  // the staging's last store has read it
                __syncwarp();
#pragma unroll
                for (int pn = 0; pn < NT / 64; ++pn) {
                    uint32_t v[32];
                    tmem_ld32(lo_ + kTmHi + 32 * pn, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(stage2 + pn * 4096 + swz(lane, i)) =
                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
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
                if constexpr (kStore) {  // pairs of tokens: u, then err
                    unsigned char *st = half ? stage1 : stage0;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        *reinterpret_cast<uint16_t *>(st + (2 * i) * 64 + 2 * lane) = (uint16_t)(o[i] & 0xffffu);
                        *reinterpret_cast<uint16_t *>(st + (2 * i + 1) * 64 + 2 * lane) = (uint16_t)(o[i] >> 16);
                    }
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

template <int NT, bool PAIR, bool kStore>
cudaError_t launch(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    CUtensorMap tk, tq, tx, t0, t1, ts;
    const int64_t nc = (p.L + kC - 1) / kC;
    if (!encode_4d(&tk, p.Bm, p.N, p.G, p.L, p.B, kC) || !encode_4d(&tq, p.Cm, p.N, p.G, p.L, p.B, kC) ||
        !encode_4d(&tx, p.x, p.P, p.H, p.L, p.B, kC) ||
        !encode_out(&t0, kStore ? ch.u : p.y, p.P, p.H, p.L, p.B) || !encode_out(&t1, kStore ? ch.err : p.y, p.P, p.H, p.L, p.B))
        return cudaErrorInvalidValue;
    if (kStore ? !encode_states(&ts, ch.states, p.N, p.P, p.B * p.H * nc) : (ts = t0, false)) return cudaErrorInvalidValue;
    const int tiles = PAIR ? 1 : (int)((p.P + 127) / 128);
    const int64_t streams = streams_of(p);
    const int grid = delta_tc_grid(p);
    const ChainArgs a{p.h0,   ch.prep,   ch.prep_bytes, (int)nc,  (int)p.H,  (int)p.P,        (int)p.G, (int)p.N,
                      tiles,  (int)streams, p.h_final,  ch.hand, ch.flags, ch.status, wait_limit_us()};
    constexpr int smem = Lay<NT, PAIR, kStore>::bytes;
    const auto kernel = k_delta_tc<NT, PAIR, kStore>;
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
    cfg.numAttrs = streams > grid ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, tk, tq, tx, t0, t1, ts, a);
}

template <int NT, bool kStore>
cudaError_t launch_pair(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    return pairs(p) ? launch<NT, true, kStore>(p, ch, s) : launch<NT, false, kStore>(p, ch, s);
}

}  // namespace

// One CTA per SM (it takes all of TMEM), or per stream where there are fewer.
int delta_tc_grid(const DeltaProblem &p) {
    const int sms = num_sms() > 0 ? num_sms() : 148;
    const int64_t streams = streams_of(p);
    return (int)(streams < sms ? streams : sms);
}

size_t delta_tc_hand_bytes(const DeltaProblem &p) {
    const int grid = delta_tc_grid(p);
    return streams_of(p) > grid ? (size_t)grid * 128 * (p.N <= 64 ? 64 : 128) * sizeof(float) : 0;
}

cudaError_t delta_tc_chain(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s) {
    const bool store = ch.states != nullptr;
    if (p.N <= 64) return store ? launch_pair<64, true>(p, ch, s) : launch_pair<64, false>(p, ch, s);
    return store ? launch_pair<128, true>(p, ch, s) : launch_pair<128, false>(p, ch, s);
}

}  // namespace ssd
