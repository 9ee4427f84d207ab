// decode.cuh — attention of one new token per sequence over a paged key-value
// cache, split over the cache's length and joined:
//     y_t = scale q . k_t  (t < len),  lse = log sum_t exp(y_t),
//     o   = sum_t exp(y_t - lse) v_t,
//     mass_out[t] = mass[t] + sum over the group's heads of exp(y_t - lse).
//
// Slot t of sequence b lives in page table[b][t / page], slot t % page of it;
// the pages' strides are the caller's (head-major or token-major pages, or a
// contiguous cache as one long page a sequence).
//
// The work is the cache's bytes (4 d a token and key head, against 4 d flops a
// byte-pair and query head), so the kernel is a stream of asynchronous copies:
//  - The lengths are on the device and may differ by orders of magnitude, so
//    the grid is fixed and every CTA takes an equal run of 64-token tiles out of
//    the flattened list (sequence, key head, 16-head block, tile).  A run that
//    covers a whole row of tiles writes its result; the others leave partial
//    states (maximum, sum, output), which the finish kernel folds in a fixed
//    order: results are the same run to run.  Where the table has no room for
//    long sequences, a CTA takes a whole row and there is nothing to fold.
//  - Each warp streams its own 16 tokens of every tile through its own ring of
//    shared memory (cp.async, no barrier between warps) and keeps its own
//    online softmax state; the four warps are folded at the end of a run.
//  - The query heads of a key head's group are the 16 rows of an m16n8k16
//    product (padded rows cost tensor time that a memory-bound kernel has to
//    spare); the probabilities' accumulator layout is the second product's
//    operand layout, so they never leave registers.
// Measured (bf16, d = 128, 32 heads over 8): 329 us for 4 caches of 131 thousand
// tokens on inputs in turn, 6.5 TB/s, the rate of a plain copy; 32 us for 24 ragged
// ones of 200 thousand token rows in all (with weights), where the starts of rows count.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "sm100.cuh"

namespace skl {

struct PageView {                   // a paged tensor [pages, Hk, page, d], strides in elements, d contiguous
    const void *ptr;
    long long s_page, s_head, s_slot;
};

struct DecodeParams {
    int B, H, Hk, G, nhb;           // nhb: blocks of 16 query heads per key head
    int pages, page, max_pages;     // pages in the cache, slots in a page, columns of the table
    int cap;                        // slots a sequence may have: min(max_pages * page, mass columns)
    const void *q;                  // [B, H, d]
    long long q_b, q_h;
    PageView k, v;
    const int *table, *len;
    long long table_b;              // row stride of the table
    float c;                        // scale * log2(e)
    void *o;                        // [B, H, d] contiguous
    float *lse;                     // [B, H]
    float *part_o, *part_ml;        // [2 grid][16][d], [2 grid][16][2]
    float *logits;                  // [B, H, cap] log2 units (mass wanted), or null
    const float *mass;              // [B, Hk, mass_cap]
    float *mass_out;
    int mass_cap;
    int grid;                       // CTAs of the split kernel
    int row_cost;                   // a row's start-up, in units of tiles
    int by_row;                     // one CTA a row of tiles, no partial states
    uint32_t *word;
};

constexpr int kDecTile = 64, kDecWarps = 4;

template <int D>
struct DecCfg {
    static constexpr int ROW = D * 2;
    static constexpr int STAGE = 16 * ROW * 2;                      // K and V rows of 16 tokens
    static constexpr int NSTAGE = D == 128 ? 3 : 4;
    static constexpr int RING = kDecWarps * NSTAGE * STAGE;
    static constexpr int MERGE = kDecWarps * 16 * (D + 2) * 4;      // the warps' states, after the ring is drained
    static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

// A weight enters its product with V as two 16-bit parts, hi + lo, each part a
// product of its own.  One part of 8 (bf16) or 11 (fp16) bits is off by as much as
// the rounding of the output is, and made its error against 64 bits a quarter larger;
// with two the weight is off by at most 2^-14.9 (bf16) or 2^-20.4 (fp16), and the
// output's own rounding is what is left.  The second product costs caches of
// 131 thousand tokens nothing, and short rows 5 to 8 % (24 ragged sequences 29.2 -> 31.0
// us, 7 of up to 2500 tokens 14.3 -> 15.1, one of 77 3.8 -> 4.1); the second parts in the
// product's unused rows, for up to 8 heads, brought 0.4 us of that back and were left out.
// bf16 has fp32's range; fp16 loses bits below 2^-14, so its weights are scaled to
// at most 2^15 (the scale cancels against the sum): hi has its 11 bits down to 2^-29
// of the largest.
template <typename T>
constexpr float kWeightLog2 = std::is_same<T, __half>::value ? 15.f : 0.f;

// The parts of two weights p >= 0, as operands.  hi is rounded towards zero from
// slightly below p, so that neither part of a weight is zero or negative (fp16: of
// one above 2^-29 of the largest): an infinite value stays what it is.
template <typename T>
__device__ __forceinline__ void split16(float p0, float p1, uint32_t &hi, uint32_t &lo);
template <>
__device__ __forceinline__ void split16<__nv_bfloat16>(float p0, float p1, uint32_t &hi, uint32_t &lo) {
    constexpr float kBelow = 1.f - 1.f / 65536.f;
    const uint32_t h0 = __float_as_uint(p0 * kBelow) & 0xffff0000u, h1 = __float_as_uint(p1 * kBelow) & 0xffff0000u;
    hi = __byte_perm(h0, h1, 0x7632);
    lo = pack_bf16(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1));
}
template <>
__device__ __forceinline__ void split16<__half>(float p0, float p1, uint32_t &hi, uint32_t &lo) {
    constexpr float kBelow = 1.f - 1.f / 2048.f;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1 * kBelow), "f"(p0 * kBelow));
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(p1 - h.y), "f"(p0 - h.x));
}

// D += A B, 16 x 8 x 16, fp32 accumulation.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// 16 bytes to shared memory, zeros where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Slots of sequence b: its length clamped to [0, cap] (reported if outside).
__device__ __forceinline__ int cache_len(const int *len, int b, int cap, uint32_t *word, bool report) {
    const int n = __ldg(len + b);
    if (report && (n < 0 || n > cap) && word) atomicOr(word, (uint32_t)kStatusBadLength);
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// The flattened list counts units: a row of tiles (sequence, key head, head
// block) is p.row_cost units of start-up (page table, queries, first copies,
// the fold at its end) and one unit a tile, so that a CTA with many short rows
// gets no more time's worth than one with a piece of a long row.
__device__ __forceinline__ int row_tiles(int n) { return (n + kDecTile - 1) / kDecTile; }
__device__ __forceinline__ int seq_units(int n, const DecodeParams &p) {
    return n > 0 ? (row_tiles(n) + p.row_cost) * p.Hk * p.nhb : 0;
}
__device__ __forceinline__ int run_length(int total, int grid) {
    return total > 0 ? (total + grid - 1) / grid : 1;
}

// Where a CTA of the split kernel starts: the sequence that holds its first
// unit, and the units before it.
struct RunStart {
    int total, base;
    int b, n;
};

// All threads of a block of W warps call it: a prefix sum of the sequences'
// units, 32 W sequences at a time (twice when there are more, first for the total).
template <int W>
__device__ __forceinline__ RunStart run_start(const DecodeParams &p, int *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    RunStart r;
    r.total = 0;
    r.base = 0;
    r.b = -1;
    const int rounds = (p.B + 32 * W - 1) / (32 * W);
    for (int pass = rounds > 1 ? 0 : 1; pass < 2; ++pass) {
        int done = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32 * W) {
            const int b = b0 + (int)threadIdx.x;
            const int n = b < p.B ? cache_len(p.len, b, p.cap, p.word, blockIdx.x == 0) : 0;
            const int t = seq_units(n, p);
            int v = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            if (lane == 31) sh[warp] = v;
            if (threadIdx.x == 0) sh[W] = -1;
            __syncthreads();
            int first = done + v - t;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w < warp) first += sh[w];
                done += sh[w];
            }
            if (rounds == 1) r.total = done;
            if (pass == 1) {
                const int u = (int)blockIdx.x * run_length(r.total, p.grid);
                if (u >= first && u < first + t) {
                    sh[W] = b;
                    sh[W + 1] = first;
                    sh[W + 2] = n;
                }
                __syncthreads();
                if (sh[W] >= 0) {
                    r.b = sh[W];
                    r.base = sh[W + 1];
                    r.n = sh[W + 2];
                    break;
                }
            }
            __syncthreads();
        }
        if (pass == 0) r.total = done;
    }
    __syncthreads();
    return r;
}

// ROW: a CTA a row of tiles; else equal runs of the flattened list.
template <typename T, int D, bool ROW>
__global__ void __launch_bounds__(kDecWarps * 32, 2) streamkl_decode_kernel(const DecodeParams p) {
    using C = DecCfg<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sh[kDecWarps + 3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, c4 = lane & 3;                     // accumulator row and column pair

    grid_release();
    int b, n;
    int u = 0, u_end = 1, u_first = 0, base = 0;                 // units
    if constexpr (ROW) {
        b = (int)(blockIdx.x / (p.Hk * p.nhb));
        n = cache_len(p.len, b, p.cap, p.word, blockIdx.x % (p.Hk * p.nhb) == 0);
    } else {
        const RunStart rs = run_start<kDecWarps>(p, sh);
        const int chunk = run_length(rs.total, p.grid);
        u = u_first = (int)blockIdx.x * chunk;
        u_end = min(rs.total, u + chunk);
        if (u >= u_end) return;
        b = rs.b;
        n = rs.n;
        base = rs.base;
    }
    while (u < u_end) {
        const int nt = row_tiles(n);
        int item, t0, t1;                                        // (key head, head block), tiles of it
        int row_end;
        if constexpr (ROW) {
            item = (int)(blockIdx.x % (p.Hk * p.nhb));
            t0 = 0;
            t1 = nt;
            row_end = u_end;
        } else {
            item = (u - base) / (nt + p.row_cost);
            const int tiles_at = base + item * (nt + p.row_cost) + p.row_cost;
            row_end = tiles_at + nt;
            t0 = max(0, u - tiles_at);
            t1 = min(nt, max(0, u_end - tiles_at));
        }
        const int hk = item / p.nhb, hb = item % p.nhb;
        const int h0 = hk * p.G + hb * 16, nh = min(16, p.G - hb * 16);

        if (ROW || t0 < t1) {                                    // (else the run ends inside the start-up)
            // the group's query heads as the product's 16 rows (rows past nh are zero)
            uint32_t qa[D / 16][4];
            {
                const T *q = static_cast<const T *>(p.q) + (size_t)b * p.q_b + (size_t)h0 * p.q_h;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int r = g4 + (x & 1) * 8, col = kk * 16 + c4 * 2 + (x >> 1) * 8;
                        const bool in = r < nh && bound_ok(b < p.B && h0 + r < p.H, p.word, kSiteResident);
                        qa[kk][x] = in ? __ldg(reinterpret_cast<const unsigned int *>(q + r * p.q_h + col)) : 0u;
                    }
                }
            }

            // copies 16 tokens' K and V rows into a stage of this warp's ring; the
            // 16-byte chunks of a row are permuted by the row so that eight rows of
            // a column fall into different banks
            const uint32_t ring = smem_u32(smem) + warp * C::NSTAGE * C::STAGE;
            const T *kb = static_cast<const T *>(p.k.ptr) + hk * p.k.s_head;
            const T *vb = static_cast<const T *>(p.v.ptr) + hk * p.v.s_head;
            // where this warp's token t of a tile lies (lane t < 16, elements from the
            // key head's base), or -1
            struct Place { long long k, v; };
            const bool alike = p.k.s_page == p.v.s_page && p.k.s_slot == p.v.s_slot;
            auto place_of = [&](int tile) -> Place {
                const int t = tile * kDecTile + warp * 16 + (lane & 15);
                if (tile >= t1 || t >= n) return {-1, -1};
                const int at = t / p.page, slot = t - at * p.page;
                if (!bound_ok(b < p.B && at >= 0 && at < p.max_pages, p.word, kSiteTable)) return {-1, -1};
                const int pg = __ldg(p.table + (size_t)b * p.table_b + at);
                if ((unsigned)pg >= (unsigned)p.pages) {
                    if (p.word) atomicOr(p.word, (uint32_t)kStatusBadPage);
                    return {-1, -1};
                }
                if (!bound_ok(hk < p.Hk && slot >= 0 && slot < p.page, p.word, kSiteSlot)) return {-1, -1};
                const long long k = pg * p.k.s_page + slot * p.k.s_slot;
                return {k, alike ? k : pg * p.v.s_page + slot * p.v.s_slot};
            };
            auto fetch = [&](Place pl, int stage) {
                constexpr int CH = D / 8;                            // 16-byte chunks in a row
                constexpr int RPI = 32 / CH;                         // rows a warp copies at a time
                const uint32_t dst = ring + stage * C::STAGE;
                const int ch = lane % CH;
#pragma unroll
                for (int x = 0; x < 16 / RPI; ++x) {
                    const int r = x * RPI + lane / CH;
                    const long long ko = __shfl_sync(0xffffffffu, pl.k, r), vo = __shfl_sync(0xffffffffu, pl.v, r);
                    const int bytes = ko >= 0 ? 16 : 0;
                    const uint32_t at = r * C::ROW + ((ch ^ (r & 7)) << 4);
                    cp_async16(dst + at, kb + (bytes ? ko : 0) + ch * 8, bytes);
                    cp_async16(dst + 16 * C::ROW + at, vb + (bytes ? vo : 0) + ch * 8, bytes);
                }
            };

            float o[D / 8][4];
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
            float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g4 and g4 + 8

            uint32_t seen[C::NSTAGE];                                // which of the stage's 16 tokens exist
            Place next = place_of(t0);
#pragma unroll
            for (int s = 0; s < C::NSTAGE - 1; ++s) {
                const Place pl = next;
                next = place_of(t0 + s + 1);
                seen[s] = __ballot_sync(0xffffffffu, pl.k >= 0) & 0xffffu;
                if (t0 + s < t1) fetch(pl, s);
                cp_commit();
            }
            for (int tb = t0; tb < t1; tb += C::NSTAGE) {
#pragma unroll
                for (int s = 0; s < C::NSTAGE; ++s) {
                    const int tile = tb + s;
                    if (tile >= t1) break;
                    {   // the tile NSTAGE-1 ahead, into the stage that was read last
                        constexpr int A = C::NSTAGE - 1;
                        const Place pl = next;
                        const int ns = (s + A) % C::NSTAGE;
                        next = place_of(tile + A + 1);
                        seen[ns] = __ballot_sync(0xffffffffu, pl.k >= 0) & 0xffffu;
                        if (tile + A < t1) fetch(pl, ns);
                        cp_commit();
                    }
                    cp_wait<C::NSTAGE - 1>();
                    __syncwarp();
                    const uint32_t kd = ring + s * C::STAGE, vd = kd + 16 * C::ROW;
                    // logits of 16 heads x 16 tokens
                    float y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int r = (lane & 7) + ((lane >> 4) << 3), ch = kk * 2 + ((lane >> 3) & 1);
                        uint32_t kf[4];
                        ldsm4<false>(kf, kd + r * C::ROW + ((ch ^ (r & 7)) << 4));
                        mma_16816<T>(y[0], qa[kk], kf[0], kf[1]);
                        mma_16816<T>(y[1], qa[kk], kf[2], kf[3]);
                    }
                    const uint32_t live = seen[s];
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = x * 8 + c4 * 2 + (e & 1);
                            y[x][e] = (live >> tok) & 1 ? y[x][e] * p.c : -INFINITY;
                            mx[e >> 1] = fmaxf(mx[e >> 1], y[x][e]);
                        }
                    if (p.logits) {
                        const int t = tile * kDecTile + warp * 16;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (g4 + e * 8 < nh) {
                                float *dst = p.logits + ((size_t)b * p.H + h0 + g4 + e * 8) * p.cap + t;
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int z = 0; z < 2; ++z)
                                        if (t + x * 8 + c4 * 2 + z < n &&
                                            bound_ok(t + x * 8 + c4 * 2 + z < p.cap, p.word, kSitePart))
                                            dst[x * 8 + c4 * 2 + z] = y[x][e * 2 + z];
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                    }
                    const bool up = mx[0] > M[0] || mx[1] > M[1];
                    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float Mn = fmaxf(M[e], mx[e]);
                            const float a = M[e] == -INFINITY ? 0.f : ex2(M[e] - Mn);
                            l[e] *= a;
#pragma unroll
                            for (int x = 0; x < D / 8; ++x) { o[x][2 * e] *= a; o[x][2 * e + 1] *= a; }
                            M[e] = Mn;
                        }
                    }
                    uint32_t pa[4], pb[4];                           // the weights' parts
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = (M[e] == -INFINITY ? 0.f : M[e]) - kWeightLog2<T>;
                        const float p0 = ex2(y[0][2 * e] - base), p1 = ex2(y[0][2 * e + 1] - base);
                        const float p2 = ex2(y[1][2 * e] - base), p3 = ex2(y[1][2 * e + 1] - base);
                        l[e] += (p0 + p1) + (p2 + p3);
                        split16<T>(p0, p1, pa[e], pb[e]);
                        split16<T>(p2, p3, pa[e + 2], pb[e + 2]);
                    }
#pragma unroll
                    for (int dd = 0; dd < D / 16; ++dd) {
                        const int r = (lane & 7) + (((lane >> 3) & 1) << 3), ch = dd * 2 + (lane >> 4);
                        uint32_t vf[4];
                        ldsm4<true>(vf, vd + r * C::ROW + ((ch ^ (r & 7)) << 4));
                        mma_16816<T>(o[2 * dd], pa, vf[0], vf[1]);
                        mma_16816<T>(o[2 * dd + 1], pa, vf[2], vf[3]);
                        mma_16816<T>(o[2 * dd], pb, vf[0], vf[1]);
                        mma_16816<T>(o[2 * dd + 1], pb, vf[2], vf[3]);
                    }
                    __syncwarp();
                }
            }
            cp_wait<0>();
            __syncthreads();

            // fold the four warps' states
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            float *so = reinterpret_cast<float *>(smem), *sml = so + kDecWarps * 16 * D;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = warp * 16 + g4 + e * 8;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<float2 *>(so + r * D + x * 8 + c4 * 2) =
                        make_float2(o[x][2 * e], o[x][2 * e + 1]);
                if (c4 == 0) { sml[2 * r] = M[e] - kWeightLog2<T>; sml[2 * r + 1] = l[e]; }
            }
            __syncthreads();
            const bool whole = t0 == 0 && t1 == nt;
            const int slot = 2 * blockIdx.x + (u == u_first ? 0 : 1);
            for (int x = threadIdx.x; x < nh * D; x += kDecWarps * 32) {
                const int r = x / D, col = x % D;
                float Mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kDecWarps; ++w) Mx = fmaxf(Mx, sml[2 * (w * 16 + r)]);
                const float bs = Mx == -INFINITY ? 0.f : Mx;
                float sum = 0.f, lsum = 0.f;
#pragma unroll
                for (int w = 0; w < kDecWarps; ++w) {
                    const float a = ex2(sml[2 * (w * 16 + r)] - bs);
                    sum = fmaf(a, so[(w * 16 + r) * D + col], sum);
                    lsum = fmaf(a, sml[2 * (w * 16 + r) + 1], lsum);
                }
                if (!bound_ok(b < p.B && h0 + r < p.H && slot < 2 * p.grid, p.word, whole ? kSiteRowOut : kSitePart))
                    continue;
                if (whole) {
                    const float ov = lsum == 0.f ? 0.f : sum / lsum;
                    static_cast<T *>(p.o)[((size_t)b * p.H + h0 + r) * D + col] = T(ov);
                    if (col == 0)
                        p.lse[(size_t)b * p.H + h0 + r] =
                            lsum == 0.f ? -INFINITY : 0.69314718055994530942f * (bs + lg2(lsum));
                } else {
                    p.part_o[((size_t)slot * 16 + r) * D + col] = sum;
                    if (col == 0) {
                        p.part_ml[((size_t)slot * 16 + r) * 2] = Mx;
                        p.part_ml[((size_t)slot * 16 + r) * 2 + 1] = lsum;
                    }
                }
            }
            // one CTA had the whole group: its weights, from the logits just written
            if (ROW && p.mass && p.nhb == 1) {
                float *l2 = so;                                      // (the fold is done)
                __syncthreads();
                if (threadIdx.x < nh)
                    l2[threadIdx.x] = p.lse[(size_t)b * p.H + h0 + threadIdx.x] * 1.4426950408889634074f;
                __syncthreads();
                for (int t = threadIdx.x; t < p.mass_cap; t += kDecWarps * 32) {
                    const size_t at = ((size_t)b * p.Hk + hk) * p.mass_cap + t;
                    float w = 0.f;
                    if (t < n)
                        for (int r = 0; r < nh; ++r)
                            w += l2[r] == -INFINITY
                                     ? 0.f
                                     : ex2(p.logits[((size_t)b * p.H + h0 + r) * p.cap + t] - l2[r]);
                    if (t < n || p.mass_out != p.mass) p.mass_out[at] = t < n ? p.mass[at] + w : p.mass[at];
                }
            }
            __syncthreads();
        }
        u = row_end;
        if constexpr (!ROW) {
            if (u >= u_end) break;
            while (u >= base + seq_units(n, p)) {                // next sequence with tiles
                base += seq_units(n, p);
                ++b;
                n = cache_len(p.len, b, p.cap, p.word, false);
            }
        }
    }
}

// The piece of a row's units that several CTAs may share: first and last CTA,
// and where each left its partial state.
struct RowPieces {
    int start, chunk;            // first unit of the row (its start-up included)
    int c0, c1;
    __device__ __forceinline__ size_t slot(int c) const { return 2 * (size_t)c + (c * chunk >= start ? 0 : 1); }
    // (checked build) every piece lies in a run of the grid
    __device__ __forceinline__ bool ok(const DecodeParams &p) const {
        return bound_ok(c0 >= 0 && c0 <= c1 && c1 < p.grid, p.word, kSitePart);
    }
};

// A warp's sums over the sequences: all units, and those before sequence `upto`.
__device__ __forceinline__ void warp_units(const DecodeParams &p, int upto, int &total, int &before) {
    total = before = 0;
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        const int t = seq_units(cache_len(p.len, b, p.cap, p.word, false), p);
        total += t;
        if (b < upto) before += t;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    before = __reduce_add_sync(0xffffffffu, before);
}

__device__ __forceinline__ RowPieces row_pieces(const DecodeParams &p, int total, int before, int nt, int item) {
    RowPieces r;
    r.chunk = run_length(total, p.grid);
    r.start = before + item * (nt + p.row_cost);
    r.c0 = (r.start + p.row_cost) / r.chunk;
    r.c1 = (r.start + p.row_cost + nt - 1) / r.chunk;
    return r;
}

// Joint maximum and sum (log2 units) of head r of the pieces; a whole warp
// calls it and every lane gets the same bits.
__device__ __forceinline__ void join_ml(const DecodeParams &p, const RowPieces &rp, int r, float &M, float &l) {
    const int lane = threadIdx.x & 31;
    M = -INFINITY;
    for (int c = rp.c0 + lane; c <= rp.c1; c += 32) M = fmaxf(M, p.part_ml[(rp.slot(c) * 16 + r) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float bs = M == -INFINITY ? 0.f : M;
    l = 0.f;
    for (int c = rp.c0 + lane; c <= rp.c1; c += 32) {
        const float *ml = p.part_ml + (rp.slot(c) * 16 + r) * 2;
        l = fmaf(ex2(ml[0] - bs), ml[1], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
}

constexpr int kFinishTokens = 1024;     // tokens of a mass block

// After the split kernel, `n_join` blocks fold the partial states of the rows
// that several CTAs shared, a warp a (sequence, query head), in a fixed order
// (rows of empty sequences get 0 and -inf); the others add the new token's
// weights to the accumulated ones, from the saved logits.  The latter fold the
// few maxima and sums they need themselves, so the two do not wait for each other.
template <typename T, int D>
__global__ void __launch_bounds__(128) streamkl_decode_finish_kernel(const DecodeParams p, int n_join, int nx) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x < n_join) {
        const long long row = (long long)blockIdx.x * 4 + warp;
        const int b = (int)(row / p.H), h = (int)(row % p.H);
        if (b >= p.B) {
            grid_wait();
            return;
        }
        int total, before;
        warp_units(p, b, total, before);
        const int n = cache_len(p.len, b, p.cap, p.word, false), nt = row_tiles(n);
        const int hk = h / p.G, hb = (h % p.G) / 16, r = (h % p.G) % 16;
        RowPieces rp = {0, 1, 0, 0};
        if (nt > 0) rp = row_pieces(p, total, before, nt, hk * p.nhb + hb);
        grid_wait();
        constexpr int E = D / 32;
        T *o = static_cast<T *>(p.o) + (size_t)row * D + lane * E;
        if (nt == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = T(0.f);
            if (lane == 0) p.lse[row] = -INFINITY;
            return;
        }
        if (rp.c0 == rp.c1 || !rp.ok(p)) return;                 // one CTA had it whole
        float M, l;
        join_ml(p, rp, r, M, l);
        const float bs = M == -INFINITY ? 0.f : M;
        float sum[E];
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll 4
        for (int c = rp.c0; c <= rp.c1; ++c) {
            const size_t s = rp.slot(c) * 16 + r;
            const float a = ex2(p.part_ml[s * 2] - bs);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(p.part_o + s * D + lane * E + e);
                sum[e] = fmaf(a, v.x, sum[e]);
                sum[e + 1] = fmaf(a, v.y, sum[e + 1]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = T(l == 0.f ? 0.f : sum[e] / l);
        if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : 0.69314718055994530942f * (bs + lg2(l));
        return;
    }
    // weights: tokens [t0, t0 + kFinishTokens) of one (sequence, key head)
    __shared__ float l2[32];
    const int x = (int)blockIdx.x - n_join, bk = x / nx, b = bk / p.Hk, hk = bk % p.Hk;
    const int t0 = (x % nx) * kFinishTokens, t1 = min(p.mass_cap, t0 + kFinishTokens);
    const int n = cache_len(p.len, b, p.cap, p.word, false), nt = row_tiles(n);
    int total = 0, before = 0;
    if (t0 < n && !p.by_row) warp_units(p, b, total, before);
    // the split kernel writes neither of the two, so what it does not change is copied now
    constexpr int PER = kFinishTokens / 128;
    float w[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int t = t0 + k * 128 + (int)threadIdx.x;
        const size_t at = (size_t)bk * p.mass_cap + t;
        w[k] = t < t1 && (t < n || p.mass_out != p.mass) ? p.mass[at] : 0.f;
    }
    if (p.mass_out != p.mass) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int t = t0 + k * 128 + (int)threadIdx.x;
            if (t >= n && t < t1) p.mass_out[(size_t)bk * p.mass_cap + t] = w[k];
        }
    }
    grid_wait();
    if (t0 >= n) return;
    float sum[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) sum[k] = 0.f;
    for (int g0 = 0; g0 < p.G; g0 += 32) {                       // 32 heads of the group at a time
        const int ng = min(32, p.G - g0);
        for (int g = warp; g < ng; g += 4) {
            const int hb = (g0 + g) / 16, r = (g0 + g) % 16;
            RowPieces rp = {0, 1, 0, 0};
            if (!p.by_row) rp = row_pieces(p, total, before, nt, hk * p.nhb + hb);
            float v;
            if (rp.c0 == rp.c1 || !rp.ok(p)) {
                v = p.lse[(size_t)b * p.H + hk * p.G + g0 + g] * 1.4426950408889634074f;
            } else {
                float M, l;
                join_ml(p, rp, r, M, l);
                v = l == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) + lg2(l);
            }
            if (lane == 0) l2[g] = v;
        }
        __syncthreads();
        for (int g = 0; g < ng; ++g) {
            const float *y = p.logits + ((size_t)b * p.H + hk * p.G + g0 + g) * p.cap;
            const float s = l2[g];
            if (s == -INFINITY) continue;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int t = t0 + k * 128 + (int)threadIdx.x;
                if (t < n) sum[k] += ex2(y[t] - s);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int t = t0 + k * 128 + (int)threadIdx.x;
        if (t < n && t < t1) p.mass_out[(size_t)bk * p.mass_cap + t] = w[k] + sum[k];
    }
}

}  // namespace skl
