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
// The products are a few percent of what the memory takes, so the warp-level mma, whose operands
// and results are in the registers of the one warp that needs them, costs nothing against tcgen05
// and saves its round trips through tensor memory.  P enters as two bf16 parts (the outputs are
// float32), each tile's P.V starts from zero and is added in fp32, rounded to nearest.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

template <int D>
struct FewCfg {
    static constexpr int T = 16;                 // rows of a tile
    static constexpr int CH = D / 8;             // 16-byte chunks of a row
    static constexpr int TILE = T * D * 2;       // bytes of a K or V tile
    static constexpr int S = 3;                  // tiles of a warp's ring
    static constexpr int WARPS = D == 128 ? 8 : 16;
    static constexpr int SMEM_BYTES = WARPS * S * 2 * TILE;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// 16 bytes from global to shared memory; zeros when `some` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
span_few_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kc,
                const __nv_bfloat16 *__restrict__ vc, const __grid_constant__ SpanParams p) {
    using C = FewCfg<D>;
    constexpr int T = C::T, CH = C::CH, S = C::S;
    extern __shared__ __align__(128) uint8_t few_smem[];
    const int lane = threadIdx.x & 31;
    const int worker = blockIdx.x * C::WARPS + (threadIdx.x >> 5);
    const uint32_t ring = smem_u32(few_smem) + (threadIdx.x >> 5) * (S * 2 * C::TILE);

    // Behind the launch over the shared rows nothing here depends on it: what that launch waited for
    // before it let this one start is all that is read.  The launch behind this one has to find both
    // complete, so the wait comes at the end.
    if (!p.behind_shared) grid_dependency_wait();
    grid_launch_dependents();
    // in the ring, which nothing uses yet
    auto *const before = reinterpret_cast<long long *>(few_smem);
    const SpanRange cr = locate_warp_ranges<C::WARPS * 32>(p, worker, blockIdx.x == 0, before, before + C::WARPS * 32);
    __syncthreads();
    if (lane == 0) open_notes(p, worker);

    // The copies run S - 1 tiles ahead, with a walker of their own.
    SpanWalker cw;
    cw.init(p, cr);
    SpanSegment cg;
    int cj = 0;
    bool copies_left = cw.next(p, cg);
    int n_copied = 0;
    // 16-row tiles start on multiples of 8 rows of the table, so a tile has at most two pages.  Their
    // numbers are read when the copy before is issued.
    int pages[2];
    auto look_up = [&]() {
        if constexpr (PAGED) {
            const int t0 = (cg.j0 + cj) * T;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                pages[h] = copies_left && t0 + 8 * h < cg.rows
                               ? __ldg(p.block_table + static_cast<long long>(cg.src) * p.max_pages + (cg.row0 + t0 + 8 * h) / p.page_size)
                               : 0;
        }
    };
    look_up();
    auto copy_tile = [&]() {
        if (copies_left) {
            const int t0 = (cg.j0 + cj) * T, rows = cg.rows - t0;  // rows left from here on
            const uint32_t dst = ring + (n_copied % S) * (2 * C::TILE);
            long long base[2];
            if constexpr (PAGED) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = cg.row0 + t0 + 8 * h;
                    int pg = pages[h];
                    if (pg < 0 || pg >= p.n_pages) {
                        if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_PAGE_RANGE);
                        pg = 0;
                    }
                    base[h] = static_cast<long long>(pg) * p.page_size + row % p.page_size - 8 * h;
                }
            } else {
                base[0] = base[1] = static_cast<long long>(cg.src) * (cg.s < p.P ? p.g_max : p.own_max) + cg.row0 + t0;
            }
            constexpr int STEP = 32 / CH;  // rows per instruction
            const int r0 = lane / CH, c = lane % CH;
            const long long stride = static_cast<long long>(p.H_kv) * D;
#pragma unroll
            for (int i = 0; i < T / STEP; ++i) {
                const int r = i * STEP + r0;
                const bool some = r < rows;
                const long long at = some ? (base[i * STEP >= 8] + r) * stride + cg.kvh * D + c * 8 : 0;
                const uint32_t to = dst + r * (D * 2) + ((c ^ (r & 7)) << 4);
                copy16(to, kc + at, some);
                copy16(to + C::TILE, vc + at, some);
            }
            ++n_copied;
            if (++cj == cg.len) {
                copies_left = cw.next(p, cg);
                cj = 0;
            }
            look_up();
        }
        copy_commit();  // an empty group keeps the count
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy_tile();

    SpanWalker w;
    w.init(p, cr);
    SpanSegment g;
    int n = 0;
    const float neg = p.negate ? -1.f : 1.f;
    while (w.next(p, g)) {
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
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

        for (int jj = 0; jj < g.len; ++jj, ++n) {
            copy_wait<S - 2>();
            __syncwarp();  // the tile is there for everyone, and everyone has left the one before
            copy_tile();
            const uint32_t kt = ring + (n % S) * (2 * C::TILE), vt = kt + C::TILE;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                const int r = (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
                ldmatrix4(b, kt + r * (D * 2) + ((c ^ (r & 7)) << 4));
                mma(s[0], qa[k], b[0], b[1]);
                mma(s[1], qa[k], b[2], b[3]);
            }
            const int t0 = (g.j0 + jj) * T;
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
                        pr[h][x][e] = in ? s[x][2 * h + e] * (neg * p.scale_log2) : -INFINITY;
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
                        o[j][2 * h] *= alpha;
                        o[j][2 * h + 1] *= alpha;
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
                const int r = ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * j + (lane >> 4);
                ldmatrix4_t(b, vt + r * (D * 2) + ((c ^ (r & 7)) << 4));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float t[4] = {};
                    mma(t, lo, b[2 * x], b[2 * x + 1]);
                    mma(t, hi, b[2 * x], b[2 * x + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[2 * j + x][e] += t[e];
                }
            }
        }
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
                *reinterpret_cast<float2 *>(dst + 8 * j + 2 * (lane % 4)) = make_float2(o[j][2 * h] * norm, o[j][2 * h + 1] * norm);
        }
    }
    if (p.behind_shared) grid_dependency_wait();
}

namespace {

template <int D, bool PAGED>
int launch_span_few_impl(const SpanParams &p, const void *q, const void *k, const void *v, cudaStream_t stream) {
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
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
                           static_cast<const __nv_bfloat16 *>(v), p) != cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int span_few_warps(int d) { return d == 128 ? FewCfg<128>::WARPS : FewCfg<64>::WARPS; }

int launch_span_few(const SpanParams &p, const void *q, const void *k, const void *v, cudaStream_t stream) {
    if (p.block_table != nullptr)
        return p.d == 128 ? launch_span_few_impl<128, true>(p, q, k, v, stream) : launch_span_few_impl<64, true>(p, q, k, v, stream);
    return p.d == 128 ? launch_span_few_impl<128, false>(p, q, k, v, stream) : launch_span_few_impl<64, false>(p, q, k, v, stream);
}

}  // namespace gqa
