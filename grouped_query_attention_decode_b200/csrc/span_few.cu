// Few query rows (up to 16 a unit) against spans of a bf16 cache.
//
// A sequence's own rows behind those it shares, or an encoder's states under one token: every
// cached row meets a handful of query rows, so the work is the reading of K and V, and the spans
// are often short.  span_tc.cu pays a chain of waits for every unit there (load, scores, softmax,
// product, epilogue: ~5 us for a unit of 2 tiles) and the split-KV decode does too.  Here a worker
// is one warp with its own range of the line (tiles of 16 rows), its own ring of tiles, and no
// barrier with anyone; what hides the chain is the other warps of the SM.
//
//   S[16 x 16] = Q[16 x d] . K_tile^T,  O[16 x d] += P[16 x 16] . V_tile    (mma m16n8k16)
//
// The products keep the tensor pipe active a quarter of the time, so the warp-level mma, whose
// operands and results are in the registers of the one warp that needs them, is fast enough and
// saves tcgen05's round trips through tensor memory.  P enters as two bf16 parts (the outputs are
// float32), each tile's P.V starts from zero and is added in fp32, rounded to nearest.
//
// Measured (one B200): 32 sequences of 1024 states, 64/64 heads, d = 64, one token each: 537 MB in
// 110 us, 4.9 TB/s; issue slots are 42 % used, the tensor pipe 26 %, and a warp mostly waits for its
// own chain.  Short calls also pay ~6 us before the first copy.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

constexpr unsigned long long kFewDrainNs = 1000000000ull;

template <int D>
struct FewCfg {
    static constexpr int T = 16;                 // rows of a tile
    static constexpr int KB = D / 64;            // 128-byte column blocks of a row
    static constexpr int TILE = T * D * 2;       // bytes of a K or V tile: KB blocks of 16 rows of 128 bytes
    static constexpr int S = 3;                  // tiles of a warp's ring
    static constexpr int WARPS = D == 128 ? 8 : 16;
    static constexpr int BOXES = 4 * KB;         // copies of a tile: K or V, 8 rows, a column block
    static constexpr int RING_BYTES = WARPS * S * 2 * TILE;
    static constexpr int BAR_BYTES = (WARPS * S * 8 + 127) / 128 * 128;
    static constexpr int SMEM_BYTES = RING_BYTES + BAR_BYTES + WARPS * 33 * 8;  // and locate_warp_ranges' sums
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}

}  // namespace

template <int D, bool PAGED>
__global__ void __launch_bounds__(FewCfg<D>::WARPS * 32, 1)
span_few_kernel(const __grid_constant__ SpanFewMaps maps,
                const __nv_bfloat16 *__restrict__ q, const __grid_constant__ SpanParams p) {
    using C = FewCfg<D>;
    constexpr int T = C::T, S = C::S, KB = C::KB;
    extern __shared__ __align__(1024) uint8_t few_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = blockIdx.x * C::WARPS + warp;
    uint8_t *const ring = few_smem + warp * (S * 2 * C::TILE);
    uint64_t *const full = reinterpret_cast<uint64_t *>(few_smem + C::RING_BYTES) + warp * S;
    if ((smem_u32(few_smem) & 1023u) != 0) {
        grid_dependency_wait();
        if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, GQA_STATUS_INTERNAL);
        return;
    }
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(full + i, 1);
        fence_mbarrier_init();
    }
    if (threadIdx.x == 0) {
        if (p.s_begin < p.P) {
            prefetch_tmap(maps.kv);
            prefetch_tmap(maps.kv + 1);
        }
        if (p.s_end > p.P) {
            prefetch_tmap(maps.kv + 2);
            prefetch_tmap(maps.kv + 3);
        }
    }

    // Behind the launch over the shared rows nothing here depends on it: what that launch waited for
    // before it let this one start is all that is read.  The launch behind this one has to find both
    // complete, so the wait comes at the end.
    if (!p.behind_shared) grid_dependency_wait();
    grid_launch_dependents();
    auto *const before = reinterpret_cast<long long *>(few_smem + C::RING_BYTES + C::BAR_BYTES);
    const SpanRange cr = locate_warp_ranges<C::WARPS * 32>(p, worker, blockIdx.x == 0, before, before + C::WARPS * 32);
    if (lane == 0) open_notes(p, worker);

    // The copies run S - 1 tiles ahead, with a walker of their own.
    SpanWalker cw;
    cw.init(p, cr);
    SpanSegment cg;
    int cj = 0;
    bool copies_left = cw.next(p, cg);
    int n_copied = 0;
    // Lane i < BOXES copies one box of a tile: K or V, a column block, its first or last 8 rows.
    // A box lies in one page (pages hold multiples of 8 rows and tiles start at multiples of 8);
    // the page's number is read when the copy before is issued.
    const bool is_v = lane & 1;
    const int cb = KB == 2 ? (lane >> 1) & 1 : 0, half = lane / (2 * KB);
    uint8_t *const to = ring + (is_v ? C::TILE : 0) + cb * 2048 + half * 1024;
    const uint64_t once = l2_policy_evict_first();
    int row, outer;  // of the box
    auto look_up = [&]() {
        if (!copies_left) return;
        const int t0 = (cg.j0 + cj) * T + 8 * half;
        row = cg.row0 + t0;
        outer = cg.src;
        if constexpr (PAGED) {
            if (lane < C::BOXES && t0 < cg.rows) {
                const int i = row / p.page_size;
                outer = __ldg(p.block_table + static_cast<long long>(cg.src) * p.max_pages + i);
                row -= i * p.page_size;
            }
        }
    };
    look_up();
    auto copy_tile = [&]() {
        if (!copies_left) return;
        const int st = n_copied % S, rows = cg.rows - (cg.j0 + cj) * T;  // rows left from the tile's first on
        if (lane == 0) mbar_arrive_expect_tx(full + st, (rows > 8 ? 2 : 1) * 2 * KB * 1024);
        __syncwarp();
        if (lane < C::BOXES && 8 * half < rows) {
            if (PAGED && (outer < 0 || outer >= p.n_pages)) {
                if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_PAGE_RANGE);
                outer = 0;
            }
            // K and V of the shared rows, then of the own ones
            const CUtensorMap *tm = maps.kv + (cg.s < p.P ? 0 : 2) + is_v;
            tma_load_4d(to + st * (2 * C::TILE), tm, full + st, cb * 64, cg.kvh, row, outer, once);
        }
        ++n_copied;
        if (++cj == cg.len) {
            copies_left = cw.next(p, cg);
            cj = 0;
        }
        look_up();
    };
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) copy_tile();

    SpanWalker w;
    w.init(p, cr);
    SpanSegment g;
    int n = 0;
    bool ok = true;
    const float scale = p.negate ? -p.scale_log2 : p.scale_log2;
    // ldmatrix rows and 16-byte chunks of this lane: K as it lies (rows are the second operand's
    // columns), V transposed; chunk c of row r stands at c ^ (r % 8)
    const int kr = (lane >> 4) * 8 + (lane & 7), vr = ((lane >> 3) & 1) * 8 + (lane & 7);
    const uint32_t k_at = smem_u32(ring) + kr * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
    const uint32_t v_at = smem_u32(ring) + C::TILE + vr * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
    while (ok && w.next(p, g)) {
        if (lane == 0) note_unit(p, g, cr, worker);
        // This thread's query rows are lane / 4 and lane / 4 + 8; its q values, as the first operand
        // of the score product, are columns 16 k + 2 (lane % 4) .. + 1 and + 8 of both.
        long long orow[2];
        int seen[2];
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int token;
            orow[h] = span_row(p, g, 0, lane / 4 + 8 * h, token);
            seen[h] = orow[h] >= 0 ? seen_rows(p, g, token) : 0;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(q + (orow[h] >= 0 ? orow[h] : 0) * D) + lane % 4;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][h] = orow[h] >= 0 ? __ldg(src + 8 * k) : 0u;
                qa[k][h + 2] = orow[h] >= 0 ? __ldg(src + 8 * k + 4) : 0u;
            }
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float2 o[D / 8][2];  // [8 columns][row]
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = make_float2(0.f, 0.f);

        for (int jj = 0; jj < g.len; ++jj, ++n) {
            const int st = n % S;
            ok = __all_sync(kFullMask, wait_bounded(full + st, (n / S) & 1, nullptr, p.wait_ns));
            if (!ok) break;
            copy_tile();  // into the slot of the tile before, which everyone has left
            const uint32_t off = st * (2 * C::TILE);
            const int t0 = (g.j0 + jj) * T;
            if (g.rows - t0 < T) {
                // rows past the end: their weights are 0, but what stands there may be NaN or infinite
                for (int i = (g.rows - t0) * 8 + lane; i < T * 8; i += 32)
#pragma unroll
                    for (int b = 0; b < KB; ++b)
                        *reinterpret_cast<uint4 *>(ring + off + C::TILE + b * 2048 + i * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();  // before a later copy into the slot
                __syncwarp();
            }
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldmatrix4(b, (k_at + off + (k >> 2) * 2048) ^ ((k & 3) << 5));
                mma(s[0], qa[k], b[0], b[1]);
                mma(s[1], qa[k], b[2], b[3]);
            }
            float pr[2][2][2];  // [row][8 columns][value]
            bool raise = false;
            float m_new[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool in = t0 + 8 * x + 2 * (lane & 3) + e < seen[h];
                        pr[h][x][e] = in ? s[x][2 * h + e] * scale : -INFINITY;
                        top = fmaxf(top, pr[h][x][e]);
                    }
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
                m_new[h] = fmaxf(m[h], top);
                raise |= m_new[h] > m[h];
            }
            if (__any_sync(kFullMask, raise)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float alpha = m_new[h] == -INFINITY ? 1.f : ex2_approx(m[h] - m_new[h]);
                    m[h] = m_new[h];
                    l[h] *= alpha;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][h].x *= alpha;
                        o[j][h].y *= alpha;
                    }
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float a = ex2_approx(pr[h][x][0] - ref), b = ex2_approx(pr[h][x][1] - ref);
                    l[h] += a + b;
                    hi[2 * x + h] = pack_bf16(a, b);
                    lo[2 * x + h] = pack_bf16(a - __uint_as_float(hi[2 * x + h] << 16), b - __uint_as_float(hi[2 * x + h] & 0xffff0000u));
                }
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t b[4];
                ldmatrix4_t(b, (v_at + off + (j >> 2) * 2048) ^ ((j & 3) << 5));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float t[4] = {};
                    mma(t, lo, b[2 * x], b[2 * x + 1]);
                    mma(t, hi, b[2 * x], b[2 * x + 1]);
                    o[2 * j + x][0] = add_f32x2(o[2 * j + x][0], make_float2(t[0], t[1]));
                    o[2 * j + x][1] = add_f32x2(o[2 * j + x][1], make_float2(t[2], t[3]));
                }
            }
        }
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
            l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (orow[h] < 0) continue;
            const int row = lane / 4 + 8 * h;
            float *dst, *ml = nullptr;
            float norm = 1.f;
            if (!g.whole()) {
                float *slot = p.slots + (2ll * worker + (g.first ? 0 : 1)) * p.slot_floats;
                dst = slot + row * D;
                ml = slot + p.unit_rows * D + 2 * row;
            } else if (p.B > 0) {
                const long long rr = (g.s < p.P ? 0 : static_cast<long long>(p.N) * p.H_q) + orow[h];
                dst = p.res + rr * D;
                ml = p.res_ml + 2 * rr;
            } else {
                dst = p.out + orow[h] * D;
                norm = 1.f / l[h];
            }
            if (ml != nullptr && lane % 4 == 0) *reinterpret_cast<float2 *>(ml) = make_float2(m[h], l[h]);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2 *>(dst + 8 * j + 2 * (lane % 4)) = make_float2(o[j][h].x * norm, o[j][h].y * norm);
        }
    }
    if (!ok) {
        if (lane == 0 && p.status != nullptr) atomicOr(p.status, GQA_STATUS_WAIT_TIMEOUT);
        // no copy may still be writing this CTA's shared memory when it exits
        for (int i = n; i < n_copied; ++i) wait_bounded(full + i % S, (i / S) & 1, nullptr, kFewDrainNs);
    }
    if (p.behind_shared) grid_dependency_wait();
}

namespace {

template <int D, bool PAGED>
int launch_span_few_impl(const SpanParams &p, const SpanFewMaps &maps, const void *q, cudaStream_t stream) {
    using C = FewCfg<D>;
    auto kern = span_few_kernel<D, PAGED>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GQA_ERR_CUDA;
    if (dev < 64 && !attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
            return GQA_ERR_CUDA;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.G + C::WARPS - 1) / C::WARPS);
    cfg.blockDim = dim3(C::WARPS * 32);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, maps, static_cast<const __nv_bfloat16 *>(q), p) != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int span_few_warps(int d) { return d == 128 ? FewCfg<128>::WARPS : FewCfg<64>::WARPS; }

int launch_span_few(const SpanParams &p, const SpanFewMaps &maps, const void *q, cudaStream_t stream) {
    if (p.block_table != nullptr)
        return p.d == 128 ? launch_span_few_impl<128, true>(p, maps, q, stream) : launch_span_few_impl<64, true>(p, maps, q, stream);
    return p.d == 128 ? launch_span_few_impl<128, false>(p, maps, q, stream) : launch_span_few_impl<64, false>(p, maps, q, stream);
}

}  // namespace gqa
