// mass.cuh — column sums of one softmax matrix: the attention weight that each
// key has received from a set of query rows,
//     lse_i  = log sum_j exp(y_ij),   y_ij = scale q_i . k_j  (visible j)
//     mass_j = sum_{heads of the group} sum_i exp(y_ij - lse_i)
// without writing the matrix.  Both sums run in one kernel template:
//   MODE = kRowLse: a CTA owns 128 query rows and streams the keys.  The rows
//          are the (query head, row) pairs of one key head's group, packed, so
//          that a few rows of several heads fill a tile.
//   MODE = kKeyMass: a CTA owns 128 keys of one key head and streams the query
//          rows of all heads of its group.
// The owned rows are the MMA's M dimension (tensor-memory lanes), the streamed
// ones its N dimension, so in both modes a thread reads one owned row of a
// logit tile and its sum over the streamed rows stays in the thread.
//
// Roles (2 + 8 warps, two CTAs per SM so that one's start and end overlap the
// other's tiles):
//   warp 0   producer: TMA loads of 64 streamed rows into an NSTAGE ring; in
//            kKeyMass also the rows' -lse * log2(e), as a table beside the tile.
//   warp 1   MMA issuer and owner of the tensor memory: the owned rows sit in
//            tensor memory as the A operand (packed 16-bit), so each
//            tcgen05.mma reads only the streamed tile from shared memory.
//   warps 2..9  two warpgroups taking the logit tiles in turn; thread = owned row.
// Work bound: one exponential a pair (16 a clock and SM) against 2 d flops.
#pragma once

#include "sm100.cuh"

namespace skl {

enum StatMode { kRowLse = 0, kKeyMass = 1 };

struct StatParams {
    int B, H, Hk, G;             // G = H / Hk query heads per key head
    int N_Q, N_K, causal;
    int n_own;                   // tiles of 128 owned rows per (batch, key head)
    int splits;                  // pieces of the streamed range per owned tile
    const int *kv_len;           // per-batch key lengths, or null
    float c;                     // scale * log2(e)
    uint32_t idesc;              // instruction descriptor (bf16 or fp16 operands)
    const void *own;             // owned rows: queries or keys
    long long own_b, own_h, own_n;   // their strides in elements
    float *lse;                  // [B, H, N_Q]: written (kRowLse) or read (kKeyMass)
    float *mass;                 // [B, Hk, N_K]
    int accumulate;              // add to mass instead of overwriting it
    float *part;                 // splits > 1: partial results, one plane per split
    DevStatus st;
};

template <int D>
struct StatCfg {
    static constexpr int BM = 128, BN = 64;
    static constexpr int BOX = BN * 128;                      // one [64 rows][64 columns] 16-bit box
    static constexpr int STAGE_BYTES = BN * D * 2;
    static constexpr int NSTAGE = 4;
    static constexpr int NBUF = 3;                            // logit buffers of 64 columns
    static constexpr uint32_t TMEM_A = NBUF * BN;             // the owned rows, packed
    static constexpr uint32_t TMEM_COLS = 256;
    static constexpr int SMEM = NSTAGE * STAGE_BYTES + 1024;
    static constexpr int NWG = 2;
    static constexpr int THREADS = 64 + 128 * NWG;
    static_assert(TMEM_A + D / 2 <= TMEM_COLS, "logit buffers and the owned rows fit");
};

// 4-D tiled load: c0 = 0 or 64 columns, c1 = first row, c2 = head, c3 = batch.
__device__ __forceinline__ void tma_load_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                              int c3, int n0, int n1, int n2, int n3, uint32_t *word) {
    if (!bound_ok(c0 >= 0 && (c0 & 63) == 0 && c0 + 64 <= n0 && c1 >= 0 && c1 < n1 && c2 >= 0 && c2 < n2 && c3 >= 0 &&
                      c3 < n3,
                  word, kSiteTma))
        return;
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// mbar_wait by a whole warp, whose lanes take the same way out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const DevStatus &st, volatile int *abort_flag,
                                          uint32_t who) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort_flag, who));
}

// Online log-sum-exp state of one row: M the running maximum (log2 units), l
// the sum of 2^(y - M).  One chunk of 32 raw logits; hidden ones are -inf.
__device__ __forceinline__ void lse_chunk(const float (&u)[32], float c, float &M, float &l) {
    float m0 = fmax3(u[0], u[1], u[2]), m1 = fmax3(u[3], u[4], u[5]);
#pragma unroll
    for (int k = 6; k < 30; k += 4) {
        m0 = fmax3(m0, u[k], u[k + 1]);
        m1 = fmax3(m1, u[k + 2], u[k + 3]);
    }
    const float cm = fmax3(m0, m1, fmaxf(u[30], u[31])) * c;
    // the running maximum may lag by 8 (terms up to 2^8 are as exact), which
    // saves the rescaling of the sum for most chunks
    if (!__all_sync(0xffffffffu, cm <= M + 8.f)) {
        const float Mn = fmaxf(M, cm);
        l *= M == -INFINITY ? 0.f : ex2(M - Mn);
        M = Mn;
    }
    const float base = M == -INFINITY ? 0.f : M;    // nothing visible yet: every term is 2^-inf
    const uint64_t c2 = f2splat(c), nM = f2splat(-base);
    uint64_t s[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        const int j = (k >> 1) & 1;
        s[j] = f2add(s[j], ex2_pair(f2fma(f2pack(u[k], u[k + 1]), c2, nM)));
    }
    const float2 t = f2unpack(f2add(s[0], s[1]));
    l += t.x + t.y;
}

// Sum over 32 streamed rows of 2^(u c + nb): nb = -lse * log2(e) of each row.
__device__ __forceinline__ float mass_chunk(const float (&u)[32], float c, const float *nb) {
    const uint64_t c2 = f2splat(c);
    uint64_t s[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        const float4 b = ld_shared_v4(nb + k);
        s[0] = f2add(s[0], ex2_pair(f2fma(f2pack(u[k], u[k + 1]), c2, f2pack(b.x, b.y))));
        s[1] = f2add(s[1], ex2_pair(f2fma(f2pack(u[k + 2], u[k + 3]), c2, f2pack(b.z, b.w))));
    }
    const float2 t = f2unpack(f2add(s[0], s[1]));
    return t.x + t.y;
}

// The same with rows to leave out: those above `first` see this key (causal),
// and a row with nb = -inf (no visible key) adds nothing whatever it holds.
__device__ __forceinline__ float mass_chunk_masked(const float (&u)[32], float c, const float *nb, int first) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const float b = nb[k];
        const float e = ex2(fmaf(u[k], c, b));
        s[k & 1] += (k >= first && b != -INFINITY) ? e : 0.f;
    }
    return s[0] + s[1];
}

template <int D, int MODE>
__global__ void __launch_bounds__(StatCfg<D>::THREADS, 2)
    streamkl_stat_kernel(const __grid_constant__ CUtensorMap mS, const StatParams p) {
    using C = StatCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sT = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    __shared__ uint64_t bar_a, bar_full[C::NSTAGE], bar_empty[C::NSTAGE], bar_sfull[C::NBUF], bar_sempty[C::NBUF];
    __shared__ uint64_t bar_quiet;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ __align__(16) float table[C::NSTAGE][C::BN];   // kKeyMass: -lse * log2(e) of the stage's rows
    __shared__ int odd[C::NSTAGE];                            // kKeyMass: some row of the stage is left out
    __shared__ float merge[2][C::BM];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // item: owned tile (the causal mask's heaviest first), split, (batch, key head)
    const int BHk = p.B * p.Hk;
    const int bk = (int)(blockIdx.x % BHk), lin = (int)(blockIdx.x / BHk);
    const int split = lin % p.splits, tile = lin / p.splits;
    const int b = bk / p.Hk, hk = bk % p.Hk;
    const int own0 = (MODE == kRowLse ? p.n_own - 1 - tile : tile) * C::BM;
    const int off = p.N_K - p.N_Q;
    const int nk = key_count(p.kv_len, b, p.N_K, p.st.word, threadIdx.x == 0 && split == 0 && tile == 0);

    // Streamed tiles of this item.  kRowLse: key tiles up to the last visible
    // key.  kKeyMass: for each head of the group the row tiles from the first
    // row that sees the tile's first key.
    int s_first = 0, s_per, n_all;
    if (MODE == kRowLse) {
        int kend = nk;
        if (p.causal) {
            // rows are packed (head, row): a tile that crosses a head's end reaches the last row
            const int r0 = own0 % p.N_Q, r1 = r0 + C::BM - 1;
            kend = min(nk, min(r1, p.N_Q - 1) + off + 1);
        }
        s_per = (kend + C::BN - 1) / C::BN;
        n_all = s_per;
    } else {
        if (p.causal) s_first = max(0, own0 - off) / C::BN;
        s_per = max(0, (p.N_Q + C::BN - 1) / C::BN - s_first);
        n_all = own0 < nk ? s_per * p.G : 0;
    }
    const int t_lo = (int)((long long)n_all * split / p.splits);
    const int n_t = (int)((long long)n_all * (split + 1) / p.splits) - t_lo;

    if (threadIdx.x == 0) {
        mbar_init(&bar_a, 4 * C::NWG);
        for (int s = 0; s < C::NSTAGE; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], MODE == kKeyMass ? 1 + 4 : 1);   // the MMA's commit, and the table's readers
        }
        for (int s = 0; s < C::NBUF; ++s) {
            mbar_init(&bar_sfull[s], 1);
            mbar_init(&bar_sempty[s], 4);
        }
        mbar_init(&bar_quiet, 1);
        abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&mS);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    volatile int *abort_v = &abort_flag;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int issued = 0;
        for (int t = 0; t < n_t; ++t) {
            const int s = t % C::NSTAGE, n = t / C::NSTAGE, u = t_lo + t;
            const int g = MODE == kKeyMass ? u / s_per : 0;
            const int row0 = (MODE == kKeyMass ? s_first + u % s_per : u) * C::BN;
            const int head = MODE == kKeyMass ? hk * p.G + g : hk;
            float nb0 = -INFINITY, nb1 = -INFINITY;
            bool out = false;
            if (MODE == kKeyMass) {
                const float *l = p.lse + ((size_t)b * p.H + head) * p.N_Q;
                const bool in = bound_ok(b < p.B && head < p.H && row0 >= 0, p.st.word, kSiteConst);
                if (in && row0 + lane < p.N_Q) {
                    nb0 = -1.4426950408889634074f * ld_now(l + row0 + lane);
                    if (fabsf(nb0) == INFINITY) { nb0 = -INFINITY; out = true; }
                }
                if (in && row0 + 32 + lane < p.N_Q) {
                    nb1 = -1.4426950408889634074f * ld_now(l + row0 + 32 + lane);
                    if (fabsf(nb1) == INFINITY) { nb1 = -INFINITY; out = true; }
                }
                out = __any_sync(0xffffffffu, out);
            }
            if (n > 0 && !warp_wait(&bar_empty[s], (n - 1) & 1, p.st, abort_v, 1)) break;
            if (MODE == kKeyMass) {
                table[s][lane] = nb0;
                table[s][lane + 32] = nb1;
                if (lane == 0) odd[s] = out;
                __syncwarp();
            }
            if (lane == 0) {
                uint8_t *dst = sT + s * C::STAGE_BYTES;
                mbar_expect_tx(&bar_full[s], C::STAGE_BYTES);
                const int nh = MODE == kKeyMass ? p.H : p.Hk, nr = MODE == kKeyMass ? p.N_Q : p.N_K;
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_rows(dst + x * C::BOX, &mS, &bar_full[s], x * 64, row0, head, b, D, nr, nh, p.B,
                                  p.st.word);
            }
            issued = t + 1;
        }
        if (*abort_v && lane == 0) {
            // copies in flight land before the CTA's memory is released
            DevStatus quick = p.st;
            quick.budget_ns = 50000000ull;
            volatile int never = 0;
            for (int t = (issued > C::NSTAGE ? issued - C::NSTAGE : 0); t < issued; ++t)
                mbar_wait(&bar_full[t % C::NSTAGE], (t / C::NSTAGE) & 1, quick, &never, 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint64_t d0 = sw128_desc(smem_u32(sT), 16, 1024);
        if (elect_one()) {
            if (n_t > 0 && mbar_wait(&bar_a, 0, p.st, abort_v, 2)) {
                for (int t = 0; t < n_t; ++t) {
                    const int s = t % C::NSTAGE, buf = t % C::NBUF, use = t / C::NBUF;
                    if (!mbar_wait(&bar_full[s], (t / C::NSTAGE) & 1, p.st, abort_v, 3)) break;
                    if (use > 0 && !mbar_wait(&bar_sempty[buf], (use - 1) & 1, p.st, abort_v, 4)) break;
                    tc_fence_after();
                    const uint64_t ds = desc_add(d0, s * C::STAGE_BYTES);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16_ts(tmem + buf * C::BN, tmem + C::TMEM_A + kk * 8,
                                    desc_add(ds, (kk >> 2) * C::BOX + (kk & 3) * 32), p.idesc, kk > 0);
                    mma_commit(&bar_sfull[buf]);
                    mma_commit(&bar_empty[s]);
                }
            }
            mma_quiesce(&bar_quiet, p.st, 9);
        }
    } else {
        // ------------------------------------------------------------ owned rows
        const int wg = (warp - 2) >> 2, sub = warp & 3, row = sub * 32 + lane;
        const int orow = own0 + row;                          // packed query row, or key
        const uint32_t lane_base = tmem + ((uint32_t)(sub * 32) << 16);
        const int n_rows = MODE == kRowLse ? p.G * p.N_Q : p.N_K;
        const int g = MODE == kRowLse ? orow / p.N_Q : 0, i = MODE == kRowLse ? orow - g * p.N_Q : orow;
        if (n_t > 0) {
            // this warpgroup's half of its rows into tensor memory
            const int h = MODE == kRowLse ? hk * p.G + g : hk;
            const bool in = orow < n_rows && bound_ok(b < p.B && h < (MODE == kRowLse ? p.H : p.Hk) && i >= 0 &&
                                                          i < (MODE == kRowLse ? p.N_Q : p.N_K),
                                                      p.st.word, kSiteResident);
            const __nv_bfloat16 *src = in ? static_cast<const __nv_bfloat16 *>(p.own) + b * p.own_b + h * p.own_h +
                                                i * p.own_n + wg * (D / 2)
                                          : nullptr;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                row_to_tmem<16>(lane_base + C::TMEM_A + wg * (D / 4) + x * 16, src ? src + x * 32 : nullptr);
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_a);

        float M = -INFINITY, l = 0.f, mass = 0.f;
        for (int t = wg; t < n_t; t += 2) {
            const int buf = t % C::NBUF, s = t % C::NSTAGE, u = t_lo + t;
            const int row0 = (MODE == kKeyMass ? s_first + u % s_per : u) * C::BN;
            if (!warp_wait(&bar_sfull[buf], (t / C::NBUF) & 1, p.st, abort_v, 5)) break;
            // the table's rows were written before the stage's barrier filled
            if (MODE == kKeyMass && !warp_wait(&bar_full[s], (t / C::NSTAGE) & 1, p.st, abort_v, 6)) break;
            tc_fence_after();
            float tile_sum = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v[32];
                tmem_ld32(lane_base + buf * C::BN + x * 32, v);
                tmem_ld_wait();
                const int c0 = row0 + x * 32;
                if (MODE == kRowLse) {
                    const int lim = p.causal ? min(nk, i + off + 1) : nk;   // first hidden key
                    if (!__all_sync(0xffffffffu, c0 + 32 <= lim)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (c0 + k >= lim) v[k] = -INFINITY;
                    }
                    lse_chunk(v, p.c, M, l);
                } else {
                    // row i sees key j iff i >= j - off
                    const int first = p.causal ? orow - off - c0 : 0;
                    if (odd[s] || !__all_sync(0xffffffffu, first <= 0))
                        tile_sum += mass_chunk_masked(v, p.c, &table[s][x * 32], first);
                    else
                        tile_sum += mass_chunk(v, p.c, &table[s][x * 32]);
                }
            }
            mass += tile_sum;     // tile by tile: a long sum's rounding grows with its number of terms
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar_sempty[buf]);
                if (MODE == kKeyMass) mbar_arrive(&bar_empty[s]);
            }
        }
        // the two warpgroups' halves of each row
        if (wg == 1) {
            if (MODE == kRowLse) {
                merge[0][row] = M;
                merge[1][row] = l;
            } else {
                merge[0][row] = mass;
            }
        }
        named_sync(1, 128 * C::NWG);
        if (wg == 0 && orow < n_rows && !*abort_v) {
            if (MODE == kRowLse) {
                const float M1 = merge[0][row], l1 = merge[1][row];
                const float Mn = fmaxf(M, M1);
                l = (M == -INFINITY ? l : l * ex2(M - Mn)) + (M1 == -INFINITY ? l1 : l1 * ex2(M1 - Mn));
                const size_t r = ((size_t)b * p.H + hk * p.G + g) * p.N_Q + i;
                if (bound_ok(hk * p.G + g < p.H && i < p.N_Q, p.st.word, kSiteRowOut)) {
                    if (p.splits > 1) {
                        const size_t rows = (size_t)p.B * p.H * p.N_Q;
                        float *q = p.part + (size_t)split * 2 * rows + r;
                        q[0] = Mn;
                        q[rows] = l;
                    } else {
                        p.lse[r] = l == 0.f ? -INFINITY : 0.69314718055994530942f * ((Mn == -INFINITY ? 0.f : Mn) + lg2(l));
                    }
                }
            } else {
                // keys at and past the batch element's length received nothing
                const float m = orow < nk ? mass + merge[0][row] : 0.f;
                const size_t r = (size_t)bk * p.N_K + orow;
                if (p.splits > 1)
                    p.part[(size_t)split * BHk * p.N_K + r] = m;
                else
                    p.mass[r] = p.accumulate ? p.mass[r] + m : m;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the splits' states of each row in a fixed order.
__global__ void __launch_bounds__(256) streamkl_lse_merge_kernel(const float *__restrict__ part, int splits,
                                                                 long long rows, float *__restrict__ lse) {
    const long long r = (long long)blockIdx.x * 256 + threadIdx.x;
    if (r >= rows) return;
    float M = -INFINITY;
    for (int s = 0; s < splits; ++s) M = fmaxf(M, part[(size_t)s * 2 * rows + r]);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int s = 0; s < splits; ++s)
        l += part[((size_t)s * 2 + 1) * rows + r] *
             (part[(size_t)s * 2 * rows + r] == -INFINITY ? 1.f : ex2(part[(size_t)s * 2 * rows + r] - base));
    lse[r] = l == 0.f ? -INFINITY : 0.69314718055994530942f * (base + lg2(l));
}

// Sums the splits' partial masses of each key in a fixed order.
__global__ void __launch_bounds__(256) streamkl_mass_sum_kernel(const float *__restrict__ part, int splits,
                                                                long long n, int accumulate, float *__restrict__ mass) {
    const long long r = (long long)blockIdx.x * 256 + threadIdx.x;
    if (r >= n) return;
    float m = 0.f;
    for (int s = 0; s < splits; ++s) m += part[(size_t)s * n + r];
    mass[r] = accumulate ? mass[r] + m : m;
}

}  // namespace skl
