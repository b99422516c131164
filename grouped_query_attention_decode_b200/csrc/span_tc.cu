// Groups of query rows against spans of a bf16 cache, on sm_100a tensor cores (tcgen05 + TMA).
//
// The attention of a batch that shares rows (gqa_decode_shared*) and of tokens over an encoder's
// states (gqa_cross_attend).  One persistent CTA per SM walks its range of tiles (spans.cuh).
// The query rows of a unit -- (token, query head of the group) pairs -- are the M dimension, so a
// cached tile is read once for up to 256 rows:
//
//   S[128 rows x 128] = Q[128 x d] . K_tile^T       (UMMA, both operands in shared memory)
//   softmax, online across tiles, one query row per thread, in fp32
//   O[128 rows x d]  += P[128 x 128] . V_tile       (UMMA, P in tensor memory)
//
// The outputs are float32, so P enters the second product as two bf16 parts (high, and what the
// rounding left), two products of 128 each: ~16 significant bits instead of 8, for 1.5 times the
// tensor work.  P overwrites its S tile in place: the 32 columns of 32 scores become 16 columns of
// packed high parts and 16 of low parts.  O stays in tensor memory over all tiles; a row is
// rescaled there only when its maximum grows by more than kLazyLog2.
//
// Work of a CTA is one sequence of steps, a step being one row tile against one cached tile, and
// step z belongs to stream z & 1: each stream has its own S/P and O in tensor memory and its own
// softmax warpgroup, so the tensor cores work on one stream while the other's softmax runs.  A
// unit of two row tiles alternates them over each cached tile (K and V are loaded once for both);
// a unit of one row tile alternates its cached tiles between the streams, which are joined when
// the piece ends.  Issue order: S(z+1) goes before P.V(z), so a stream's next scores are ready as
// soon as its P has been used; tcgen05.mma of one thread execute in order, so S(z+2) may overwrite
// the P of step z right behind P.V(z).
// Roles (384 threads):
//   warp 0      TMA producer (q tiles, K and V tiles), also owns the tensor memory
//   warp 1      UMMA issuer (one elected thread)
//   warp 2      zeroes the rows past a span's end in its last V tile
//   warp 3      idle
//   warps 4..11 two softmax / rescale / epilogue warpgroups
// Every wait is bounded; on a timeout the CTA drains its copies and UMMAs, frees its tensor
// memory, sets GQA_STATUS_WAIT_TIMEOUT and returns.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

constexpr unsigned long long kSpanDrainNs = 1000000000ull;
constexpr float kSpanLazyLog2 = 8.0f;  // as in the decode kernel

template <int D>
struct SpanCfg {
    static constexpr int T = 128, RT = 128;
    static constexpr int KB = D / 64;             // 128-byte column blocks of a row
    static constexpr int TILE_BYTES = T * D * 2;  // one K, V or q tile
    static constexpr int THREADS = 384;
    static constexpr int S = D == 128 ? 5 : 10;   // ring slots, one K or V tile each
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t O_COL = 256;        // S/P of stream x at 128 x, O at 256 + D x
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128, false, false);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
    static constexpr uint32_t NEGATE_A = 1u << 13;
    struct Small {
        uint64_t full[S], empty[S], fixed[S];
        uint64_t q_full[2], q_empty[2];
        uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
        uint64_t ml_full[2][4];  // per stream and warp: its rows' (m, l) are in ml
        uint64_t mma_done;
        SpanRange range;
        long long scratch[THREADS / 32];
        uint32_t tmem_base;
        int abort;
        float2 ml[2][RT];  // (m, l) of each stream's rows when a piece ends
    };
    static constexpr int SMEM_BYTES = (2 + S) * TILE_BYTES + static_cast<int>(sizeof(Small));
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// One step of a CTA's range.
struct Step {
    SpanSegment g;
    int jj, steps;  // step within the segment, steps of the segment
    bool pair;      // two row tiles per cached tile

    __device__ bool open(const SpanParams &p, SpanWalker &w) {
        if (!w.next(p, g)) return false;
        jj = 0;
        pair = g.ntok > p.tb;
        steps = pair ? 2 * g.len : g.len;
        return true;
    }
    __device__ int tile() const { return g.j0 + (pair ? jj >> 1 : jj); }
    __device__ int rows(const SpanParams &p) const { return min(p.T, g.rows - tile() * p.T); }
    // the step is the first (last) of its segment to use its cached tile
    __device__ bool takes() const { return !pair || (jj & 1) == 0; }
    __device__ bool gives() const { return !pair || (jj & 1) == 1; }
    // ... to use its q tile
    __device__ bool takes_q() const { return jj < (pair ? 2 : 1); }
    __device__ bool gives_q() const { return jj >= steps - (pair ? 2 : 1); }
};

// Runs s(step) and pv(step) for every step in issue order: S(z+1) before P.V(z).  Both return
// false to stop.
template <class FS, class FP>
__device__ __forceinline__ bool for_each_op(const SpanParams &p, const SpanRange &cr, FS s, FP pv) {
    SpanWalker w;
    w.init(p, cr);
    Step cur, prev;
    bool more = cur.open(p, w);
    if (!more) return true;
    if (!s(cur)) return false;
    while (more) {
        prev = cur;
        more = ++cur.jj < cur.steps || cur.open(p, w);
        if (more && !s(cur)) return false;
        if (!pv(prev)) return false;
    }
    return true;
}

}  // namespace

template <int D, bool PAGED>
__global__ void __launch_bounds__(SpanCfg<D>::THREADS, 1)
span_tc_kernel(const __grid_constant__ SpanMaps maps, const __grid_constant__ SpanParams p) {
    using C = SpanCfg<D>;
    constexpr int T = C::T, S = C::S;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *const q_base = smem;
    uint8_t *const ring = smem + 2 * C::TILE_BYTES;
    auto *const sm = reinterpret_cast<typename C::Small *>(ring + S * C::TILE_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, GQA_STATUS_INTERNAL);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 2);  // the issuer's use of the slot and warp 2's look at it
            mbar_init(&sm->fixed[s], 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&sm->q_full[j], 1);
            mbar_init(&sm->q_empty[j], 1);
            mbar_init(&sm->s_full[j], 1);
            mbar_init(&sm->p_full[j], 4);
            mbar_init(&sm->o_full[j], 1);
            mbar_init(&sm->o_empty[j], 8);
            for (int w = 0; w < 4; ++w) mbar_init(&sm->ml_full[j][w], 1);
        }
        mbar_init(&sm->mma_done, 1);
        sm->abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&sm->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    // Everything below reads what the kernels before on the stream wrote.
    grid_dependency_wait();
    tc_fence_before_sync();
    locate_span_range<C::THREADS>(p, blockIdx.x, sm->scratch, &sm->range);
    tc_fence_after_sync();
    grid_launch_dependents();

    const uint32_t tmem = sm->tmem_base;
    const SpanRange cr = sm->range;
    volatile int *abort_flag = &sm->abort;
    const uint64_t budget = p.wait_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_WAIT_TIMEOUT);
    };

    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer
        const uint64_t once = l2_policy_evict_first();   // rows that one unit reads
        const uint64_t again = l2_policy_evict_normal();  // rows that several units read
        int n = 0, nq = 0;  // ring slots and q tiles filled
        // A K (or V) tile of the cursor's step into the next ring slot.
        auto load = [&](const Step &c, bool v) {
            const SpanSegment &g = c.g;
            const bool shared = g.s < p.P;
            const int row0 = g.row0 + c.tile() * T, rows = c.rows(p);
            const bool fulltile = rows == T;
            const int boxr = !fulltile ? 8 : PAGED ? min(p.page_size, T) : T;
            const int nbox = fulltile ? T / boxr : (rows + 7) >> 3;
            int pg = g.src, row = row0 + lane * boxr;
            if constexpr (PAGED) {
                if (lane < nbox) {
                    pg = __ldg(p.block_table + static_cast<long long>(g.src) * p.max_pages + row / p.page_size);
                    if (pg < 0 || pg >= p.n_pages) {
                        if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_PAGE_RANGE);
                        pg = 0;
                    }
                    row %= p.page_size;
                }
            }
            const int st = n % S;
            bool got = true;
            if (lane == 0 && n >= S) got = wait_bounded(&sm->empty[st], ((n / S) - 1) & 1, abort_flag, budget);
            if (!__shfl_sync(kFullMask, got, 0)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&sm->full[st], C::KB * nbox * boxr * 128);
            __syncwarp();
            if (lane < nbox) {
                const CUtensorMap *m =
                    shared ? (v ? (fulltile ? &maps.v_shared : &maps.v_shared8) : (fulltile ? &maps.k_shared : &maps.k_shared8))
                           : (v ? (fulltile ? &maps.v_own : &maps.v_own8) : (fulltile ? &maps.k_own : &maps.k_own8));
                uint8_t *dst = ring + st * C::TILE_BYTES + lane * boxr * 128;
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb)
                    tma_load_4d(dst + kb * T * 128, m, &sm->full[st], kb * 64, g.kvh, row, pg, shared ? again : once);
            }
            ++n;
            return true;
        };
        const bool ok = for_each_op(
            p, cr,
            [&](const Step &c) {
                if (c.takes_q()) {
                    const int qb = nq & 1;
                    bool got = true;
                    if (lane == 0 && nq >= 2) got = wait_bounded(&sm->q_empty[qb], ((nq >> 1) - 1) & 1, abort_flag, budget);
                    if (!__shfl_sync(kFullMask, got, 0)) return false;
                    if (lane == 0) {
                        const SpanSegment &g = c.g;
                        const bool shared = g.s < p.P;
                        const int toks = shared ? p.tb : min(p.tb, p.Q);
                        mbar_arrive_expect_tx(&sm->q_full[qb], C::KB * toks * p.rb * 128);
#pragma unroll
                        for (int kb = 0; kb < C::KB; ++kb)
                            tma_load_3d(q_base + qb * C::TILE_BYTES + kb * C::RT * 128, shared ? &maps.q_shared : &maps.q_own,
                                        &sm->q_full[qb], kb * 64, g.kvh * p.r + g.hb * p.rb, g.tok0 + c.jj * p.tb);
                    }
                    ++nq;
                }
                return !c.takes() || load(c, false);
            },
            [&](const Step &c) { return !c.takes() || load(c, true); });
        if (lane == 0) {
            if (!ok) fail();
            // no copy may still be writing this CTA's shared memory when it exits
            for (int i = n > S ? n - S : 0; i < n; ++i) wait_bounded(&sm->full[i % S], (i / S) & 1, nullptr, kSpanDrainNs);
            for (int i = nq > 2 ? nq - 2 : 0; i < nq; ++i) wait_bounded(&sm->q_full[i & 1], (i >> 1) & 1, nullptr, kSpanDrainNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ UMMA issuer
        if (lane == 0) {
            // K and q: K-major, 8-row groups 1024 B apart.  V: MN-major (d by rows), its 64-column
            // blocks T * 128 B apart.
            const uint64_t dk0 = sdesc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t dv0 = sdesc_sw128(smem_u32(ring), T * 128, 1024);
            const uint64_t dq0 = sdesc_sw128(smem_u32(q_base), 16, 1024);
            const uint32_t idesc_qk = C::IDESC_QK | (p.negate ? C::NEGATE_A : 0u);
            int n = 0;           // ring slots taken
            int zs = 0, zp = 0;  // steps whose S (P.V) was issued
            int nq = 0, qbase = 0;  // q tiles taken, q tile of the segment's first step
            int kslot = 0, vslot = 0;
            int uses[2] = {0, 0};    // segments each stream took part in
            uint32_t fixes = 0;      // per slot: parity of its next `fixed` phase
            const bool ok = for_each_op(
                p, cr,
                [&](const Step &c) {
                    if (c.jj == 0) qbase = nq;
                    if (c.takes_q()) {
                        if (!wait_bounded(&sm->q_full[nq & 1], (nq >> 1) & 1, abort_flag, budget)) return false;
                        ++nq;
                    }
                    if (c.takes()) {
                        kslot = n % S;
                        if (!wait_bounded(&sm->full[kslot], (n / S) & 1, abort_flag, budget)) return false;
                        ++n;
                    }
                    const int qb = (qbase + (c.pair ? c.jj & 1 : 0)) & 1;
                    tc_fence_after_sync();
                    const uint64_t dq = dq0 + ((qb * C::TILE_BYTES) >> 4), dk = dk0 + ((kslot * C::TILE_BYTES) >> 4);
                    const uint32_t dst = tmem + (zs & 1) * 128;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * T * 128 + (kk & 3) * 32) >> 4;
                        umma_bf16(dst, dq + off, dk + off, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&sm->s_full[zs & 1]);
                    if (c.gives()) umma_commit(&sm->empty[kslot]);
                    if (c.gives_q()) umma_commit(&sm->q_empty[qb]);
                    ++zs;
                    return true;
                },
                [&](const Step &c) {
                    const int x = zp & 1;
                    if (c.takes()) {
                        vslot = n % S;
                        if (!wait_bounded(&sm->full[vslot], (n / S) & 1, abort_flag, budget)) return false;
                        ++n;
                        if (c.rows(p) < T) {
                            if (!wait_bounded(&sm->fixed[vslot], (fixes >> vslot) & 1u, abort_flag, budget)) return false;
                            fixes ^= 1u << vslot;
                        }
                    }
                    if (c.jj < 2) {  // the stream's first step of the segment: O must have been read
                        if (uses[x] > 0 && !wait_bounded(&sm->o_empty[x], (uses[x] - 1) & 1, abort_flag, budget)) return false;
                        ++uses[x];
                    }
                    if (!wait_bounded(&sm->p_full[x], (zp >> 1) & 1, abort_flag, budget)) return false;
                    tc_fence_after_sync();
                    const uint64_t dv = dv0 + ((vslot * C::TILE_BYTES) >> 4);
                    const uint32_t pt = tmem + x * 128, dst = tmem + C::O_COL + x * D;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < T / 16; ++kk)
                            umma_bf16_ts(dst, pt + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8, dv + ((kk * 2048) >> 4), C::IDESC_PV,
                                         (c.jj >= 2 || part > 0 || kk > 0) ? 1u : 0u);
                    if (c.gives()) umma_commit(&sm->empty[vslot]);
                    if (c.jj >= c.steps - 2) umma_commit(&sm->o_full[x]);
                    ++zp;
                    return true;
                });
            if (!ok) fail();
            umma_commit(&sm->mma_done);
            wait_bounded(&sm->mma_done, 0, nullptr, kSpanDrainNs);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------ V rows past the end
        // A row past the span has weight 0 in P, but what the copy brought (or left) there may
        // be NaN or infinite: zero it.  The warp sees every filling of every slot, in order, so
        // that the phases it waits for cannot run ahead of it.
        int n = 0;
        auto look = [&](const Step &c, bool v) {
            if (!c.takes()) return true;
            const int st = n % S;
            const bool got = wait_bounded(&sm->full[st], (n / S) & 1, abort_flag, budget);
            if (!__all_sync(kFullMask, got)) return false;
            ++n;
            const int rows = c.rows(p);
            if (v && rows < T) {
                uint8_t *tile = ring + st * C::TILE_BYTES;
                const int chunks = (T - rows) * 8;  // 16-byte chunks per column block
                for (int i = lane; i < chunks * C::KB; i += 32) {
                    const int kb = i / chunks, rem = i - kb * chunks;
                    *reinterpret_cast<uint4 *>(tile + kb * T * 128 + rows * 128 + rem * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->fixed[st]);
            }
            if (lane == 0) mbar_arrive(&sm->empty[st]);
            return true;
        };
        const bool ok = for_each_op(
            p, cr, [&](const Step &c) { return look(c, false); }, [&](const Step &c) { return look(c, true); });
        if (!ok && lane == 0) fail();
    } else if (warp >= 4) {
        // ------------------------------------------------------------------ softmax warpgroups
        const int x = (warp - 4) >> 2;   // this warpgroup's stream
        const int q4 = warp & 3;         // TMEM lanes this warp may access
        const int row = q4 * 32 + lane;  // row of the row tile this thread owns
        const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t st = tmem + lanes + x * 128;
        SpanWalker w;
        w.init(p, cr);
        SpanSegment g;
        int z0 = 0;           // the segment's first step
        int nstep = 0;        // steps of this stream so far
        int uses = 0, joins = 0;  // segments the stream took part in, those shared by both streams
        bool ok = true;
        if (threadIdx.x == 128) open_notes(p, cr);
        while (ok && w.next(p, g)) {
            if (threadIdx.x == 128) note_unit(p, g, cr);
            const bool pair = g.ntok > p.tb;
            const int steps = pair ? 2 * g.len : g.len;
            const int jj0 = (x ^ z0) & 1;  // this stream's first step of the segment
            z0 += steps;
            const bool part = jj0 < steps;
            int token;
            const long long orow = span_row(p, g, pair ? jj0 : 0, row, token);
            const bool busy = __any_sync(kFullMask, orow >= 0);  // warps of padding rows only keep the barriers going
            const int seen = orow >= 0 ? seen_rows(p, g, token) : 1 << 30;  // padding rows hold anything
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            for (int jj = jj0; jj < steps; jj += 2, ++nstep) {
                if (!wait_bounded(&sm->s_full[x], nstep & 1, abort_flag, budget)) ok = false;
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                tc_fence_after_sync();
                if (busy) {
                    const int left = seen - (g.j0 + (pair ? jj >> 1 : jj)) * T;  // visible columns
                    const bool cut = __any_sync(kFullMask, left < T);
                    // The scores are read twice, 64 and then 32 columns at a time: holding all 128
                    // beside the parts of P costs more registers than the launch has.
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < T; c += 64) {
                        uint32_t a[64];
                        tmem_ld32(st + c, a);
                        tmem_ld32(st + c + 32, a + 32);
                        tmem_wait_ld();
                        if (cut) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (c + e >= left) a[e] = 0xff800000u;  // -infinity
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(a[e + k]), __uint_as_float(a[e + 4 + k])));
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float m_new = top * p.scale_log2;
                    const bool raise = top > -INFINITY && m_new > m + kSpanLazyLog2;
                    if (__any_sync(kFullMask, raise)) {
                        float alpha = 1.f;
                        if (raise) {
                            alpha = ex2_approx(m - m_new);  // 0 from m = -infinity
                            m = m_new;
                        }
                        l2 = mul_f32x2(l2, make_float2(alpha, alpha));
                        if (jj >= 2) {
                            // S(z) was issued behind P.V(z-2), so O holds the stream's steps so far
                            const uint32_t ot = tmem + lanes + C::O_COL + x * D;
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(ot + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(ot + c, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : -m;
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), ref2 = make_float2(ref, ref);
#pragma unroll
                    for (int c = 0; c < T; c += 32) {
                        uint32_t a[32], hl[32];
                        tmem_ld32(st + c, a);
                        tmem_wait_ld();
                        if (cut) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c + e >= left) a[e] = 0xff800000u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 t = fma_f32x2(make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), sc2, ref2);
                            const float2 pr = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                            l2 = add_f32x2(l2, pr);
                            const __nv_bfloat162 hi = __floats2bfloat162_rn(pr.x, pr.y);
                            const uint32_t hb = *reinterpret_cast<const uint32_t *>(&hi);
                            // what the rounding left, exact in fp32
                            const __nv_bfloat162 lo = __floats2bfloat162_rn(pr.x - __uint_as_float(hb << 16), pr.y - __uint_as_float(hb & 0xffff0000u));
                            hl[e / 2] = hb;
                            hl[16 + e / 2] = *reinterpret_cast<const uint32_t *>(&lo);
                        }
                        tmem_st32(st + c, hl);
                    }
                    tmem_wait_st();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->p_full[x]);
            }
            // -------- the piece ends: O, m, l to where they belong
            if (ok && part) ok = wait_bounded(&sm->o_full[x], uses & 1, abort_flag, budget);
            ok = __all_sync(kFullMask, ok);
            if (!ok) break;
            uses += part;
            const float l = l2.x + l2.y;
            const bool both = !pair && steps >= 2;  // the streams share the rows
            float wt[2] = {1.f, 0.f}, mm = m, ll = l;  // weights of this stream's O and the other's
            if (both) {
                // Exchange (m, l) with the other stream's warp of the same rows.  Its arrival also
                // says that its O is complete, and the o_empty arrivals of both that ml was read.
                sm->ml[x][row] = make_float2(m, l);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->ml_full[x][q4]);
                ok = wait_bounded(&sm->ml_full[x ^ 1][q4], joins & 1, abort_flag, budget);
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                ++joins;
                const float2 o = sm->ml[x ^ 1][row];
                mm = fmaxf(m, o.x);
                wt[0] = m == -INFINITY ? 0.f : ex2_approx(m - mm);
                wt[1] = o.x == -INFINITY ? 0.f : ex2_approx(o.x - mm);
                ll = wt[0] * l + wt[1] * o.y;
            }
            if (part) {
                tc_fence_after_sync();
                const int c0 = both ? x * (D / 2) : 0, c1 = both ? c0 + D / 2 : D;
                const int mlc = c0 == 0;
                float *dst = nullptr;
                float norm = 1.f;
                if (orow >= 0) {
                    if (!g.whole()) {
                        float *slot = p.slots + (2ll * blockIdx.x + (g.first ? 0 : 1)) * p.slot_floats;
                        const int srow = (pair ? jj0 : 0) * C::RT + row;
                        dst = slot + srow * D;
                        if (mlc) *reinterpret_cast<float2 *>(slot + p.unit_rows * D + 2 * srow) = make_float2(mm, ll);
                    } else if (p.B > 0) {
                        const long long rr = (g.s < p.P ? 0 : static_cast<long long>(p.N) * p.H_q) + orow;
                        dst = p.res + rr * D;
                        if (mlc) *reinterpret_cast<float2 *>(p.res_ml + 2 * rr) = make_float2(mm, ll);
                    } else {
                        dst = p.out + orow * D;
                        norm = 1.f / ll;
                    }
                }
                if (busy) {
                    const uint32_t ot = tmem + lanes + C::O_COL;
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        uint32_t o[32], o2[32];
                        tmem_ld32(ot + x * D + c, o);
                        if (both) tmem_ld32(ot + (x ^ 1) * D + c, o2);
                        tmem_wait_ld();
                        if (dst != nullptr) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float v[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    v[k] = __uint_as_float(o[e + k]);
                                    if (both) {
                                        // a weight of 0 belongs to a stream that saw no row of this one: its O is not looked at
                                        v[k] = wt[0] == 0.f ? 0.f : v[k] * wt[0];
                                        if (wt[1] != 0.f) v[k] = fmaf(__uint_as_float(o2[e + k]), wt[1], v[k]);
                                    }
                                    v[k] *= norm;
                                }
                                *reinterpret_cast<float4 *>(dst + c + e) = make_float4(v[0], v[1], v[2], v[3]);
                            }
                        }
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm->o_empty[x]);
                    mbar_arrive(&sm->o_empty[both ? x ^ 1 : x]);
                }
            }
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
}

namespace {

template <int D, bool PAGED>
int launch_span_tc_impl(const SpanMaps &maps, const SpanParams &p, cudaStream_t stream) {
    using C = SpanCfg<D>;
    auto kern = span_tc_kernel<D, PAGED>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GQA_ERR_CUDA;
    if (dev < 64 && !attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
            return GQA_ERR_CUDA;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.G);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, maps, p) != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int launch_span_tc(const SpanMaps &maps, const SpanParams &p, cudaStream_t stream) {
    if (p.block_table != nullptr)
        return p.d == 128 ? launch_span_tc_impl<128, true>(maps, p, stream) : launch_span_tc_impl<64, true>(maps, p, stream);
    return p.d == 128 ? launch_span_tc_impl<128, false>(maps, p, stream) : launch_span_tc_impl<64, false>(maps, p, stream);
}

}  // namespace gqa
