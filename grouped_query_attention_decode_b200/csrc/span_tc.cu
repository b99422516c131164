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
// tensor work.  P overwrites its S tile in place: the 16 columns of 16 scores become 8 columns of
// packed high parts and 8 of low parts.
//
// Work of a CTA is one sequence of steps, a step being one row tile against one cached tile, and
// step z belongs to stream z & 1: each stream has its own S/P and O in tensor memory and its own
// softmax warps, so the tensor cores work on one stream while the other's softmax runs.  A
// unit of two row tiles alternates them over each cached tile (K and V are loaded once for both);
// a unit of one row tile alternates its cached tiles between the streams, which are joined when
// the piece ends.  Issue order: S(z+1) goes before P.V(z), so a stream's next scores are ready as
// soon as its P has been used; tcgen05.mma of one thread execute in order, so S(z+2) may overwrite
// the P of step z right behind P.V(z).
//
// The accumulation in tensor memory truncates, 16 additions a tile and row: sums kept there over 32
// tiles were off by 1e-5 of the result.  So P.V of every step starts anew, and the softmax warps
// add each tile's O to the row's sums in registers (in fp32, rounded to nearest) while the tensor
// cores work on the stream's next scores.  Their loops are short on purpose: straight code for a
// whole row is fetched more slowly than it runs (209 us instead of 143 for 512 tokens over 4096
// states, 64/8 heads, d = 128).
// Roles (384 threads):
//   warp 0      TMA producer (q tiles, K and V tiles), also owns the tensor memory
//   warp 1      UMMA issuer (one elected thread)
//   warp 2      zeroes the rows past a span's end in its last V tile
//   warp 3      planner: walks the CTA's range and hands its pieces to the other warps
//   warps 4..11 softmax, sums and epilogue: stream (warp - 4) / 4, a row a thread
// Every wait is bounded; on a timeout the CTA drains its copies and UMMAs, frees its tensor
// memory, sets GQA_STATUS_WAIT_TIMEOUT and returns.
//
// Measured (one B200): 4 x 1024 tokens over 4096 states, 64/8 heads, d = 128 take 666-690 us in a
// graph, 797-825 TFLOP/s of attention and 1.5 times that of products.  A step of 128 x 128 scores
// is ~2400 cycles where its products alone are 2060 (scores 780, bound by reading both operands from
// shared memory; P.V 1280) and a softmax warp's chain is 2465.  There a CTA has 444 steps and they
// account for the time; with a few tens of steps they do not: 8 ragged targets of up to 509 tokens
// over up to 2047 states (32/8 heads) have at most 38 a CTA, 50 us, and take 84.  About 8 us are the
// start; the rest is not attributed (a CTA has two to four pieces there, and a stream's warps finish
// one before they look at the next one's scores).  Of 4 x 128 tokens over 4096 states, 56 steps, the
// tensor pipe is active 52 % of the time, DRAM 10 %.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

constexpr unsigned long long kSpanDrainNs = 1000000000ull;
constexpr float kSpanLazyLog2 = 8.0f;  // as in the decode kernel
constexpr int kPieces = 4;             // pieces the planner may be ahead

// What the planner hands over: a piece of a unit and what follows from it.
struct SpanPiece {
    SpanSegment g;
    int steps;      // 0: there are no more pieces
    int pair;       // two row tiles per cached tile
    int last_rows;  // rows of the piece's last tile
    int once;       // no other unit reads these cached rows
};

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
        uint64_t s_full[2], p_full[2], o_full[2];
        uint64_t piece_full[kPieces], piece_empty[kPieces];
        uint64_t joined[4];  // per quadrant of rows: both streams' warps have come this far
        uint64_t mma_done;
        SpanPiece piece[kPieces];
        SpanRange range;
        long long scratch[THREADS / 32];
        uint32_t tmem_base;
        int abort;
        float2 ml[2][RT];  // (m, l) of each stream's rows when a piece of both ends
    };
    static constexpr int SMEM_BYTES = (2 + S) * TILE_BYTES + static_cast<int>(sizeof(Small));
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// The pieces in the planner's ring, as one warp (or thread) reads them.
template <class Small>
struct PieceReader {
    Small *sm;
    const volatile int *abort_flag;
    uint64_t budget;

    __device__ bool wait(int i) const {
        return wait_bounded(&sm->piece_full[i % kPieces], (i / kPieces) & 1, abort_flag, budget);
    }
    __device__ const SpanPiece &at(int i) const { return sm->piece[i % kPieces]; }
    __device__ void release(int i) const { mbar_arrive(&sm->piece_empty[i % kPieces]); }
};

// One step of a piece.
struct Step {
    int i, jj;  // piece, step within it
    int steps, pair, last_rows;

    // the step is the first (last) of its piece to use its cached tile
    __device__ bool takes() const { return !pair || (jj & 1) == 0; }
    __device__ bool gives() const { return !pair || (jj & 1) == 1; }
    // ... to use its q tile
    __device__ bool takes_q() const { return jj < (pair ? 2 : 1); }
    __device__ bool gives_q() const { return jj >= steps - (pair ? 2 : 1); }
    __device__ int tile() const { return pair ? jj >> 1 : jj; }  // within the piece
    __device__ int rows() const { return jj >= steps - (pair ? 2 : 1) ? last_rows : 128; }
};

// Runs s(step) and pv(step) for every step in issue order: S(z+1) before P.V(z).  Both return
// false to stop.  `done` releases a piece.
template <class Reader, class FS, class FP, class FD>
__device__ __forceinline__ bool for_each_op(const Reader &r, FS s, FP pv, FD done) {
    Step a, b;
    auto open = [&](Step &c, int i) {
        const SpanPiece &p = r.at(i);
        c.i = i;
        c.jj = 0;
        c.steps = p.steps;
        c.pair = p.pair;
        c.last_rows = p.last_rows;
    };
    if (!r.wait(0)) return false;
    open(a, 0);
    if (a.steps == 0) return true;
    b = a;
    if (!s(a)) return false;
    ++a.jj;
    bool more = true;
    while (true) {
        if (more) {
            if (a.jj == a.steps) {
                if (!r.wait(a.i + 1)) return false;
                open(a, a.i + 1);
                more = a.steps != 0;
            }
            if (more) {
                if (!s(a)) return false;
                ++a.jj;
            }
        }
        if (!pv(b)) return false;
        if (++b.jj == b.steps) {
            done(b.i);
            if (!more && b.i + 1 == a.i) return true;
            open(b, b.i + 1);
        }
    }
}

// A ring position and the parity of its phase.
template <int S>
struct Slot {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == S) {
            at = 0;
            phase ^= 1;
        }
    }
};

}  // namespace

template <int D, bool PAGED>
__global__ void __launch_bounds__(SpanCfg<D>::THREADS, 1)
span_tc_kernel(const __grid_constant__ SpanMaps maps, const __grid_constant__ SpanParams p) {
    using C = SpanCfg<D>;
    constexpr int T = C::T, S = C::S;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *const q_base = smem;
    uint8_t *const ring = smem + 2 * C::TILE_BYTES;
    using Small = typename C::Small;
    auto *const sm = reinterpret_cast<Small *>(ring + S * C::TILE_BYTES);
    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);  // the same in all lanes, and known to be
    const int lane = threadIdx.x & 31;

    if ((smem_u32(smem) & 1023u) != 0) {
        grid_dependency_wait();  // what is launched behind counts on it
        if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, GQA_STATUS_INTERNAL);
        return;
    }
    // a few barriers to a thread: one thread takes a thousand cycles for all of them
    const int t = threadIdx.x - 64;
    if (t >= 0 && t < S) {
        mbar_init(&sm->full[t], 1);
        mbar_init(&sm->empty[t], 2);  // the issuer's use of the slot and warp 2's look at it
        mbar_init(&sm->fixed[t], 1);
    } else if (t >= 16 && t < 18) {
        mbar_init(&sm->q_full[t - 16], 1);
        mbar_init(&sm->q_empty[t - 16], 1);
        mbar_init(&sm->s_full[t - 16], 1);
        mbar_init(&sm->p_full[t - 16], 4);
        mbar_init(&sm->o_full[t - 16], 1);
    } else if (t >= 20 && t < 20 + kPieces) {
        mbar_init(&sm->piece_full[t - 20], 1);
        mbar_init(&sm->piece_empty[t - 20], 11);  // warps 0..2 and the softmax warps
    } else if (t >= 24 && t < 28) {
        mbar_init(&sm->joined[t - 24], 2);
    } else if (t == 28) {
        mbar_init(&sm->mma_done, 1);
        sm->abort = 0;
    }
    if (t >= 0 && t < 32) fence_mbarrier_init();
    if (warp == 0) {
        tmem_alloc(&sm->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    } else if (warp == 1 && lane < 10) {
        prefetch_tmap(&maps.q_shared + lane);  // the ten of SpanMaps, in a row
    }
    // Everything below reads what the kernels before on the stream wrote.
    grid_dependency_wait();
    tc_fence_before_sync();
    locate_span_range<C::THREADS>(p, blockIdx.x, sm->scratch, &sm->range);
    tc_fence_after_sync();
    grid_launch_dependents();

    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort;
    const uint64_t budget = p.wait_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_WAIT_TIMEOUT);
    };
    const PieceReader<Small> pieces = {sm, abort_flag, budget};

    // 384 threads launch with 168 registers each; the softmax warps hold a row's sums and take more:
    // 128 * 72 + 256 * 216 = 384 * 168.  (Each branch opens with its setmaxnreg: where the two met
    // again the compiler would keep to the smaller number.)
    if (warp >= 4) {
        set_max_registers_up<216>();
        // ------------------------------------------------------------------ softmax warps
        const int x = (warp - 4) >> 2;   // this warp's stream
        const int q4 = warp & 3;         // TMEM lanes this warp may access
        const int row = q4 * 32 + lane;  // row of the row tile this thread owns
        const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t st = tmem + lanes + x * 128, ot = tmem + lanes + C::O_COL + x * D;
        uint32_t z0 = 0;       // parity of the piece's first step
        uint32_t s_phase = 0;  // parity of the stream's next scores
        uint32_t o_phase = 0;  // parity of the stream's next O
        bool ok = true;
        float2 o2[D / 2];      // the row's sums
        // Adds the O of the stream's last step to the sums.
        auto take_o = [&](bool busy) {
            const bool got = wait_bounded(&sm->o_full[x], o_phase, abort_flag, budget);
            o_phase ^= 1;
            if (!__all_sync(kFullMask, got)) return false;
            if (busy) {
                tc_fence_after_sync();
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(ot + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        o2[(c + e) / 2] = add_f32x2(o2[(c + e) / 2], make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
                }
                tc_fence_before_sync();
            }
            return true;
        };
        for (int i = 0; ok; ++i) {
            ok = __all_sync(kFullMask, pieces.wait(i));
            if (!ok) break;
            const SpanPiece &pc = pieces.at(i);
            const SpanSegment &g = pc.g;
            const int steps = pc.steps;
            if (steps == 0) break;
            const bool pair = pc.pair;
            const int jj0 = (x ^ z0) & 1;  // this stream's first step of the piece
            z0 ^= steps & 1;
            const bool both = !pair && steps >= 2;  // the streams share the rows
            // visible columns of the stream's first tile, and how many fewer from one step of the
            // stream to the next; padding rows hold anything
            int left = 1 << 30;
            {
                int token;
                if (span_row(p, g, pair ? jj0 : 0, row, token) >= 0) left = seen_rows(p, g, token) - (g.j0 + (pair ? 0 : jj0)) * T;
            }
            const bool busy = __any_sync(kFullMask, left < 1 << 30);  // warps of padding rows only keep the barriers going
            const int fewer = pair ? T : 2 * T;
            float m = -INFINITY;
            float2 l2[2] = {};
#pragma unroll
            for (int e = 0; e < D / 2; ++e) o2[e] = make_float2(0.f, 0.f);
            for (int jj = jj0; jj < steps; jj += 2, left -= fewer) {
                if (jj >= 2) {
                    ok = take_o(busy);
                    if (!ok) break;
                }
                ok = __all_sync(kFullMask, wait_bounded(&sm->s_full[x], s_phase, abort_flag, budget));
                s_phase ^= 1;
                if (!ok) break;
                if (busy) {
                    tc_fence_after_sync();
                    const bool cut = __any_sync(kFullMask, left < T);
                    // The scores are read twice: beside the sums there is no room for a whole row.
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < T; c += 64) {
                        uint32_t a[64];
                        tmem_ld32(st + c, a);
                        tmem_ld32(st + c + 32, a + 32);
                        tmem_wait_ld();
                        if (cut) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (c + e >= left) a[e] = 0xff800000u;  // -infinity
                            tmem_st32(st + c, a);
                            tmem_st32(st + c + 32, a + 32);
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(a[e + k]), __uint_as_float(a[e + 4 + k])));
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float m_new = top * p.scale_log2;
                    // The reference only has to keep the exponentials in range: it is raised when the
                    // maximum passes it by kSpanLazyLog2.
                    const bool raise = top > -INFINITY && m_new > m + kSpanLazyLog2;
                    if (__any_sync(kFullMask, raise)) {
                        float alpha = 1.f;
                        if (raise) {
                            alpha = ex2_approx(m - m_new);  // 0 from m = -infinity
                            m = m_new;
                        }
                        const float2 al2 = make_float2(alpha, alpha);
                        l2[0] = mul_f32x2(l2[0], al2);
                        l2[1] = mul_f32x2(l2[1], al2);
#pragma unroll
                        for (int e = 0; e < D / 2; ++e) o2[e] = mul_f32x2(o2[e], al2);
                    }
                    const float ref = m == -INFINITY ? 0.f : -m;
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), ref2 = make_float2(ref, ref);
#pragma unroll 1
                    for (int c = 0; c < T; c += 32) {
                        uint32_t a[32];
                        tmem_ld32(st + c, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int b = 0; b < 32; b += 16) {
                            uint32_t hl[16];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float2 t = fma_f32x2(make_float2(__uint_as_float(a[b + e]), __uint_as_float(a[b + e + 1])), sc2, ref2);
                                const float2 pr = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                                l2[(e >> 1) & 1] = add_f32x2(l2[(e >> 1) & 1], pr);
                                const __nv_bfloat162 hi = __floats2bfloat162_rn(pr.x, pr.y);
                                const uint32_t hb = *reinterpret_cast<const uint32_t *>(&hi);
                                // what the rounding left, exact in fp32
                                const float2 left2 = fma_f32x2(make_float2(__uint_as_float(hb << 16), __uint_as_float(hb & 0xffff0000u)), make_float2(-1.f, -1.f), pr);
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(left2.x, left2.y);
                                hl[e / 2] = hb;
                                hl[8 + e / 2] = *reinterpret_cast<const uint32_t *>(&lo);
                            }
                            tmem_st16(st + c + b, hl);
                        }
                    }
                    tmem_wait_st();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->p_full[x]);
            }
            if (!ok) break;
            if (jj0 >= steps) {  // a piece of one step is the other stream's
                __syncwarp();
                if (lane == 0) pieces.release(i);
                continue;
            }
            // -------- the piece ends: sums, m, l to where they belong
            ok = take_o(busy);
            if (!ok) break;
            float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
            int c0 = 0, c1 = D;
            if (both && busy) {
                // The streams share the rows.  Each finishes half of the columns and leaves the other
                // half of its sums in its O's place in tensor memory for the other stream's warp of
                // the same rows.
                sm->ml[x][row] = make_float2(m, l);
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    uint32_t v[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 t = x == 0 ? o2[(D / 2 + c + e) / 2] : o2[(c + e) / 2];
                        v[e] = __float_as_uint(t.x);
                        v[e + 1] = __float_as_uint(t.y);
                    }
                    tmem_st16(ot + c, v);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->joined[q4]);
                ok = __all_sync(kFullMask, wait_bounded(&sm->joined[q4], 0, abort_flag, budget));
                if (!ok) break;
                tc_fence_after_sync();
                const float2 other = sm->ml[x ^ 1][row];
                const float mm = fmaxf(m, other.x);
                // a stream that saw none of the row's rows weighs nothing
                const float w0 = m == -INFINITY ? 0.f : ex2_approx(m - mm), w1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - mm);
                m = mm;
                l = w0 * l + w1 * other.y;
                const uint32_t ot2 = tmem + lanes + C::O_COL + (x ^ 1) * D;
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(ot2 + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        // both streams keep what they finish in the first half of the registers
                        const float2 t = x == 0 ? o2[(c + e) / 2] : o2[(D / 2 + c + e) / 2];
                        o2[(c + e) / 2] = fma_f32x2(t, make_float2(w0, w0), mul_f32x2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), make_float2(w1, w1)));
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                // the second phase: all have read
                if (lane == 0) mbar_arrive(&sm->joined[q4]);
                ok = __all_sync(kFullMask, wait_bounded(&sm->joined[q4], 1, abort_flag, budget));
                if (!ok) break;
                c0 = x * (D / 2);
                c1 = c0 + D / 2;
            }
            // Where the row goes: looked up again, the registers being short meanwhile.
            int token;
            const long long orow = span_row(p, g, pair ? jj0 : 0, row, token);
            const bool whole = g.whole();
            float *dst = nullptr, *dst_ml = nullptr;
            if (orow >= 0) {
                if (!whole) {
                    float *slot = p.slots + (2ll * blockIdx.x + (g.first ? 0 : 1)) * p.slot_floats;
                    const int srow = (pair ? jj0 : 0) * C::RT + row;
                    dst = slot + srow * D;
                    dst_ml = slot + p.unit_rows * D + 2 * srow;
                } else if (p.B > 0) {
                    const long long rr = (g.s < p.P ? 0 : static_cast<long long>(p.N) * p.H_q) + orow;
                    dst = p.res + rr * D;
                    dst_ml = p.res_ml + 2 * rr;
                } else {
                    dst = p.out + orow * D;
                }
            }
            __syncwarp();
            if (lane == 0) pieces.release(i);
            if (dst != nullptr) {
                if (dst_ml != nullptr && c0 == 0) *reinterpret_cast<float2 *>(dst_ml) = make_float2(m, l);
                const float norm = whole && p.B == 0 ? 1.f / l : 1.f;
                dst += c0;
                // A thread writes its own row, so every store instruction touches 32 lines, which is
                // what it costs: 32 bytes at a time where the row is aligned (the workspace is; out
                // may not be).
                const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
                for (int c = 0; c < D; c += 8)
                    if (c < c1 - c0) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            v[e] = o2[(c + e) / 2].x * norm;
                            v[e + 1] = o2[(c + e) / 2].y * norm;
                        }
                        if (wide) {
                            st_global_v8(dst + c, v);
                        } else {
                            *reinterpret_cast<float4 *>(dst + c) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4 *>(dst + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
            }
        }
        if (!ok && lane == 0) fail();
    } else {
    set_max_registers_down<72>();
    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer
        const uint64_t once = l2_policy_evict_first();   // rows that one unit reads
        const uint64_t again = l2_policy_evict_normal();  // rows that several units read
        int n = 0, nq = 0;  // ring slots and q tiles filled
        // A K (or V) tile of the step into the next ring slot.
        auto load = [&](const Step &c, bool v) {
            const SpanSegment &g = pieces.at(c.i).g;
            const bool shared = g.s < p.P;
            const int row0 = g.row0 + (g.j0 + c.tile()) * T, rows = c.rows();
            const bool fulltile = rows == T;
            const int boxr = !fulltile ? 8 : PAGED ? min(p.page_size, T) : T;
            const int nbox = fulltile ? T / boxr : (rows + 7) >> 3;
            const int kvh = g.kvh;
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
                    tma_load_4d(dst + kb * T * 128, m, &sm->full[st], kb * 64, kvh, row, pg, pieces.at(c.i).once ? once : again);
            }
            ++n;
            return true;
        };
        const bool ok = for_each_op(
            pieces,
            [&](const Step &c) {
                if (c.takes_q()) {
                    const int qb = nq & 1;
                    bool got = true;
                    if (lane == 0 && nq >= 2) got = wait_bounded(&sm->q_empty[qb], ((nq >> 1) - 1) & 1, abort_flag, budget);
                    if (!__shfl_sync(kFullMask, got, 0)) return false;
                    if (lane == 0) {
                        const SpanSegment &g = pieces.at(c.i).g;
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
            [&](const Step &c) { return !c.takes() || load(c, true); },
            [&](int i) {
                __syncwarp();
                if (lane == 0) pieces.release(i);
            });
        if (lane == 0) {
            if (!ok) fail();
            // no copy may still be writing this CTA's shared memory when it exits
            for (int i = n > S ? n - S : 0; i < n; ++i) wait_bounded(&sm->full[i % S], (i / S) & 1, nullptr, kSpanDrainNs);
            for (int i = nq > 2 ? nq - 2 : 0; i < nq; ++i) wait_bounded(&sm->q_full[i & 1], (i >> 1) & 1, nullptr, kSpanDrainNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ UMMA issuer
        if (elect_one()) {
            // K and q: K-major, 8-row groups 1024 B apart.  V: MN-major (d by rows), its 64-column
            // blocks T * 128 B apart.
            const uint64_t dk0 = sdesc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t dv0 = sdesc_sw128(smem_u32(ring), T * 128, 1024);
            const uint64_t dq0 = sdesc_sw128(smem_u32(q_base), 16, 1024);
            const uint32_t idesc_qk = C::IDESC_QK | (p.negate ? C::NEGATE_A : 0u);
            Slot<S> slot;               // next ring slot
            uint32_t xs = 0, xp = 0;    // stream of the next S (P.V)
            uint32_t p_phase = 0;       // phase of p_full of step z: (z >> 1) & 1
            Slot<2> q;                  // next q tile
            int qbase = 0;              // buffer of the piece's first q tile
            uint32_t kslot = 0, vslot = 0;
            uint32_t fixes = 0;           // per slot: parity of its next `fixed` phase
            const bool ok = for_each_op(
                pieces,
                [&](const Step &c) {
                    if (c.takes_q()) {
                        if (c.jj == 0) qbase = q.at;
                        if (!wait_bounded(&sm->q_full[q.at], q.phase, abort_flag, budget)) return false;
                        q.next();
                    }
                    if (c.takes()) {
                        kslot = slot.at;
                        if (!wait_bounded(&sm->full[kslot], slot.phase, abort_flag, budget)) return false;
                        slot.next();
                    }
                    const int qb = c.pair ? (qbase ^ c.jj) & 1 : qbase;
                    tc_fence_after_sync();
                    const uint64_t dq = dq0 + ((qb * C::TILE_BYTES) >> 4), dk = dk0 + ((kslot * C::TILE_BYTES) >> 4);
                    const uint32_t dst = tmem + xs * 128;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * T * 128 + (kk & 3) * 32) >> 4;
                        umma_bf16(dst, dq + off, dk + off, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&sm->s_full[xs]);
                    if (c.gives()) umma_commit(&sm->empty[kslot]);
                    if (c.gives_q()) umma_commit(&sm->q_empty[qb]);
                    xs ^= 1;
                    return true;
                },
                [&](const Step &c) {
                    const uint32_t x = xp;
                    if (c.takes()) {
                        vslot = slot.at;
                        if (!wait_bounded(&sm->full[vslot], slot.phase, abort_flag, budget)) return false;
                        slot.next();
                        if (c.rows() < T) {
                            if (!wait_bounded(&sm->fixed[vslot], (fixes >> vslot) & 1u, abort_flag, budget)) return false;
                            fixes ^= 1u << vslot;
                        }
                    }
                    // also says that the stream's O before has been read
                    if (!wait_bounded(&sm->p_full[x], p_phase, abort_flag, budget)) return false;
                    tc_fence_after_sync();
                    const uint64_t dv = dv0 + ((vslot * C::TILE_BYTES) >> 4);
                    const uint32_t pt = tmem + x * 128, dst = tmem + C::O_COL + x * D;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < T / 16; ++kk)
                            umma_bf16_ts(dst, pt + kk * 16 + part * 8, dv + ((kk * 2048) >> 4), C::IDESC_PV,
                                         (part > 0 || kk > 0) ? 1u : 0u);
                    if (c.gives()) umma_commit(&sm->empty[vslot]);
                    umma_commit(&sm->o_full[x]);
                    p_phase ^= xp;
                    xp ^= 1;
                    return true;
                },
                [&](int i) { pieces.release(i); });
            if (!ok) fail();
            umma_commit(&sm->mma_done);
            wait_bounded(&sm->mma_done, 0, nullptr, kSpanDrainNs);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------ V rows past the end
        // A row past the span has weight 0 in P, but what the copy brought (or left) there may
        // be NaN or infinite: zero it.  The warp sees every filling of every slot, in order, so
        // that the phases it waits for cannot run ahead of it.
        Slot<S> slot;
        auto look = [&](const Step &c, bool v) {
            if (!c.takes()) return true;
            const int st = slot.at;
            const bool got = wait_bounded(&sm->full[st], slot.phase, abort_flag, budget);
            if (!__all_sync(kFullMask, got)) return false;
            slot.next();
            const int rows = c.rows();
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
            pieces, [&](const Step &c) { return look(c, false); }, [&](const Step &c) { return look(c, true); },
            [&](int i) {
                __syncwarp();
                if (lane == 0) pieces.release(i);
            });
        if (!ok && lane == 0) fail();
    } else if (warp == 3) {
        // ------------------------------------------------------------------ planner
        if (lane == 0) {
            const SpanRange cr = sm->range;
            open_notes(p, blockIdx.x);
            SpanWalker w;
            w.init(p, cr);
            SpanPiece piece;
            bool more = true, ok = true;
            for (int i = 0; more && ok; ++i) {
                more = w.next(p, piece.g);
                piece.pair = piece.last_rows = piece.steps = 0;
                if (more) {
                    piece.once = w.nblk == 1 && p.HB == 1;
                    piece.pair = piece.g.ntok > p.tb;
                    piece.steps = piece.pair ? 2 * piece.g.len : piece.g.len;
                    piece.last_rows = min(T, piece.g.rows - (piece.g.j0 + piece.g.len - 1) * T);
                }
                if (i >= kPieces) ok = wait_bounded(&sm->piece_empty[i % kPieces], ((i / kPieces) - 1) & 1, abort_flag, budget);
                if (ok) {
                    sm->piece[i % kPieces] = piece;
                    mbar_arrive(&sm->piece_full[i % kPieces]);
                    if (more) note_unit(p, piece.g, cr, blockIdx.x);
                }
            }
            if (!ok) fail();
        }
    }
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
