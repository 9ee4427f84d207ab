// mass.cuh — column sums of one softmax matrix: the attention weight that each
// key has received from a set of query rows,
//     lse_i  = log sum_j exp(y_ij),   y_ij = scale q_i . k_j  (visible j)
//     mass_j = sum_{heads of the group} sum_i exp(y_ij - lse_i)
// without writing the matrix.  Both sums run in one kernel template:
//   MODE = kRowLse: an item is 128 query rows, the keys are streamed.
//   MODE = kKeyMass: an item is 128 keys of one key head, the query rows of all
//          heads of its group are streamed.
// The item's rows are the MMA's M dimension (tensor-memory lanes), the streamed
// ones its N dimension, so in both modes a thread reads one owned row of a
// logit tile and its sum over the streamed rows stays in the thread.  Up to 64
// query rows a head are packed: a tile holds as many whole heads as fit.
//
// One CTA an SM.  The tiles of all items are one list, of which every CTA takes
// an equal run, so that causal, padded and few-item problems balance alike; an
// item that two runs share leaves partial sums, which the finish kernel adds in
// a fixed order (the same bits run to run).
//   warp 0      producer: TMA loads of an item's rows (two buffers) and of the
//               streamed tiles (a ring).
//   warps 1, 2  MMA issuers, one a half of the streamed tiles.  Warp 1 owns the
//               tensor memory: six 128 x 64 logit tiles of fp32 (halves), and the
//               item's rows (two buffers, packed 16-bit) as the A operand, so that
//               a tcgen05.mma reads only the streamed tile from shared memory (with
//               A in shared memory too, a tile took 870 clocks of its bandwidth
//               instead of 512).
//   warps 3..18 four warpgroups taking the halves in turn; thread = owned row.
//   warps 19..22 copy an item's rows from shared to tensor memory, an item ahead,
//               and in kKeyMass write the -lse * log2(e) of a half's rows as a table
//               for one warpgroup each (when every warp of the warpgroups did that
//               for itself, two thirds of the issued instructions were not sums).
//   warp 23     adds the warpgroups' sums of an item and writes it.
// Work bound: one exponential a pair (16 a clock and SM: 1024 clocks a tile)
// against 2 d flops (512 clocks a tile at d = 128).  One thread takes some 400
// clocks of its own for a half's waits, MMAs and commits, hence two issuers.
#pragma once

#include "sm100.cuh"

namespace skl {

enum StatMode { kRowLse = 0, kKeyMass = 1 };

struct StatParams {
    int B, H, Hk, G;             // G = H / Hk query heads per key head
    int N_Q, N_K, causal;
    int pack;                    // whole heads in a tile of query rows; 0: a tile is rows of one head
    int R;                       // tiles a head (pack = 0), or a group (pack > 0)
    int halves;                  // 1: no streamed tile has more than 64 rows
    const int *kv_len;           // per-batch key lengths, or null
    float c;                     // scale * log2(e)
    int fp16;                    // operands (both) are fp16, else bf16
    float *lse;                  // [B, H, N_Q]: written (kRowLse) or read (kKeyMass)
    float *mass;                 // [B, Hk, N_K]
    int accumulate;              // add to mass instead of overwriting it
    float *part;                 // [grid][2][128][2]: partial sums of a run's first and last item
    int grid;                    // runs
    DevStatus st;
};

template <int D>
struct StatCfg {
    static constexpr int BM = 128, BN = 128;
    static constexpr int BOX = 128 * 128;                     // [128 rows][64 columns] 16-bit
    static constexpr int TILE_BYTES = 128 * D * 2;
    static constexpr int NSTAGE = D == 128 ? 4 : 8;
    static constexpr int NBUF = 6;                            // logit tiles of half a streamed tile
    static constexpr uint32_t TMEM_A = NBUF * 64;             // the item's rows: two buffers of D / 2 columns
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr int SMEM = (2 + NSTAGE) * TILE_BYTES + 1024;
    // A warpgroup waits for a buffer's next filling after it has seen a later one
    // of the other buffers than the last filling (a barrier's parity repeats): as
    // many buffers as warpgroups at least, filled in order by each issuer.
    static constexpr int NWG = 4;
    static_assert(NBUF >= NWG, "see above");
    static constexpr int W_EPI = 3, W_LOAD = W_EPI + 4 * NWG, W_OUT = W_LOAD + 4;   // first warps of the roles
    static constexpr int NTABLE = 4;                          // tables a warpgroup
    static constexpr int NSLOT = 4;                           // items whose sums wait for the writer
    static constexpr int THREADS = 32 * (W_OUT + 1);
    static_assert(TMEM_A + D <= TMEM_COLS, "logit tiles and the items' rows fit");
};

// ---------------------------------------------------------------- the list of tiles
// Within one (batch, key head): `own` items, item t streaming count(t) tiles.
// With o = ceil((N_K - N_Q) / 128) (no causal mask: beyond every tile),
//   kKeyMass: key tile t is seen by row tiles max(0, t - o) .. R - 1 of each head;
//   kRowLse:  row tile r sees key tiles 0 .. min(A, r + 1 + o) - 1, A those with a key.
template <int MODE>
struct TileList {
    int own, A, o, R, mult;      // R: tiles a head; mult: heads (or packed groups of heads)
    __device__ __forceinline__ TileList(const StatParams &p, int nk) {
        A = (nk + 127) / 128;
        R = p.pack ? 1 : p.R;
        o = p.causal && !(MODE == kRowLse && p.pack) ? (p.N_K - p.N_Q + 127) / 128 : (1 << 28);
        mult = p.pack ? p.R : p.G;
        own = MODE == kKeyMass ? A : mult * R;
    }
    // r: t (kKeyMass), the tile of its head (kRowLse)
    __device__ __forceinline__ int count(int r) const {
        return MODE == kKeyMass ? mult * (R - max(0, r - o)) : min(A, r + 1 + o);
    }
    __device__ __forceinline__ long long before_row(int r) const {       // tiles of the row tiles before r of a head
        const long long x = min(max(A - 1 - o, 0), r);
        return x * (x + 1) / 2 + x * o + (r - x) * A;
    }
    __device__ __forceinline__ long long before(int t) const {           // tiles of the items before t
        if (MODE == kKeyMass) {
            const long long x = max(t - o, 0);
            return ((long long)R * t - x * (x - 1) / 2) * mult;
        }
        return (t / R) * before_row(R) + before_row(t % R);
    }
};

struct StatItem {
    int b, hk, t, nk;            // item t of (b, hk), nk keys of the batch element
    int lo, n, count;            // its tiles [lo, lo + n) of `count`
};

// Units of the whole list; a whole warp calls it.
template <int MODE>
__device__ __forceinline__ long long stat_total(const StatParams &p, bool report) {
    long long total = 0;
    if (!p.kv_len) {
        const TileList<MODE> l(p, p.N_K);
        return l.before(l.own) * p.Hk * p.B;
    }
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        const TileList<MODE> l(p, key_count(p.kv_len, b, p.N_K, p.st.word, report));
        total += l.before(l.own) * p.Hk;
    }
    for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    return total;
}

// Where unit u < total of the list falls; a whole warp calls it.
template <int MODE>
__device__ __forceinline__ void stat_find(const StatParams &p, long long u, int &b, int &hk, int &t, int &in_item) {
    if (!p.kv_len) {
        const TileList<MODE> l(p, p.N_K);
        const long long w = l.before(l.own) * p.Hk;
        b = (int)(u / w);
        u -= b * w;
    } else {
        for (int b0 = 0;; b0 += 32) {
            const int x = b0 + (int)(threadIdx.x & 31);
            long long w = 0;
            if (x < p.B) {
                const TileList<MODE> l(p, key_count(p.kv_len, x, p.N_K, p.st.word, false));
                w = l.before(l.own) * p.Hk;
            }
            long long end = w;
            for (int s = 1; s < 32; s <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, end, s);
                if ((threadIdx.x & 31) >= s) end += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, end > u);
            if (past || b0 + 32 >= p.B) {
                const int lane = past ? __ffs(past) - 1 : 31;
                b = b0 + lane;
                u -= __shfl_sync(0xffffffffu, end - w, lane);
                break;
            }
            u -= __shfl_sync(0xffffffffu, end, 31);
        }
    }
    const TileList<MODE> l(p, key_count(p.kv_len, b, p.N_K, p.st.word, false));
    const long long w = l.before(l.own);
    hk = (int)(u / w);
    u -= hk * w;
    int a = 0, z = l.own;                                     // before(a) <= u < before(z)
    while (z - a > 1) {
        const int m = (a + z) >> 1;
        if (l.before(m) <= u) a = m; else z = m;
    }
    t = a;
    in_item = (int)(u - l.before(a));
}

__device__ __forceinline__ long long stat_run(long long total, int grid) { return total > 0 ? (total + grid - 1) / grid : 1; }

// Steps through the items of a run; every role has its own copy.
template <int MODE>
struct StatIter {
    StatItem it;
    int left, r;                 // units of the run from this item on; kRowLse: the item's tile in its head
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void start(const StatParams &p, const int *rec) {
        it.b = rec[0]; it.hk = rec[1]; it.t = rec[2]; it.lo = rec[3];
        left = rec[4];
        if (left <= 0) return;
        it.nk = key_count(p.kv_len, it.b, p.N_K, p.st.word, false);
        const TileList<MODE> l(p, it.nk);
        r = MODE == kKeyMass ? it.t : it.t % l.R;
        it.count = l.count(r);
        it.n = min(it.count - it.lo, left);
    }
    __device__ __forceinline__ void next(const StatParams &p) {
        left -= it.n;
        if (left <= 0) return;
        it.lo = 0;
        ++it.t;
        ++r;
        for (;;) {
            const TileList<MODE> l(p, it.nk);
            if (r == l.R && MODE == kRowLse) r = 0;
            const bool none = it.nk == 0;                     // a batch element without keys has no tiles
            if (!none && it.t < l.own) {
                it.count = l.count(r);
                break;
            }
            it.t = 0;
            r = 0;
            if (none || ++it.hk == p.Hk) {
                it.hk = 0;
                ++it.b;
                it.nk = key_count(p.kv_len, it.b, p.N_K, p.st.word, false);
            }
        }
        it.n = min(it.count, left);
    }
};

// Query tile q of a (batch, key head): its first head and row, and its rows.
struct RowTile {
    int head, row0, rows;
};
__device__ __forceinline__ RowTile row_tile(const StatParams &p, int hk, int q) {
    RowTile r;
    if (p.pack) {
        r.head = hk * p.G + q * p.pack;
        r.row0 = 0;
        r.rows = min(p.pack, p.G - q * p.pack) * p.N_Q;
    } else {
        const int g = q / p.R;
        r.head = hk * p.G + g;
        r.row0 = (q - g * p.R) * 128;
        r.rows = min(128, p.N_Q - r.row0);
    }
    return r;
}
// The row tiles that a key tile streams, in order, without a division a tile.
struct RowCursor {
    int g, r, first;             // head of the group (packed: group of heads), tile of it, first tile that sees the keys
    __device__ __forceinline__ RowCursor(const StatParams &p, const StatItem &it, int u) {
        first = p.causal && !p.pack ? max(0, it.t - (p.N_K - p.N_Q + 127) / 128) : 0;
        const int per = p.pack ? 1 : p.R - first;
        g = per == 1 ? u : u / per;
        r = first + u - g * per;
    }
    __device__ __forceinline__ void advance(const StatParams &p, int n) {
        if (p.pack) { g += n; return; }
        r += n;
        while (r >= p.R) { r -= p.R - first; ++g; }
    }
    __device__ __forceinline__ RowTile tile(const StatParams &p, int hk) const {
        RowTile t;
        t.head = hk * p.G + (p.pack ? g * p.pack : g);
        t.row0 = p.pack ? 0 : r * 128;
        t.rows = p.pack ? min(p.pack, p.G - g * p.pack) * p.N_Q : min(128, p.N_Q - t.row0);
        return t;
    }
};

// 5-D tiled load of rows c1 .. of head c2 (and the heads after it, packed) of
// batch c4, from column 64 c3 on (one or two blocks of 64 columns a box).
__device__ __forceinline__ void tma_load_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int c1, int c2, int c3,
                                              int c4, int n1, int n2, int n3, int n4, uint32_t *word) {
    if (!bound_ok(c1 >= 0 && c1 < n1 && c2 >= 0 && c2 < n2 && c3 >= 0 && c3 < n3 && c4 >= 0 && c4 < n4, word, kSiteTma))
        return;
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// A tile of 128 rows, or (packed) of whole heads: one box, or one a block of 64 columns.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int row0, int head, int b,
                                          int rows, int pack, int n_rows, int n_heads, int n_b, uint32_t *word) {
    mbar_expect_tx(bar, rows * D * 2);
    tma_load_rows(dst, map, bar, row0, head, 0, b, n_rows, n_heads, D / 64, n_b, word);
    if (D > 64 && pack)
        tma_load_rows(dst + StatCfg<D>::BOX, map, bar, row0, head, 1, b, n_rows, n_heads, D / 64, n_b, word);
}

// mbar_wait for the long waits of this kernel's roles: the thread is suspended
// up to 10 us at a time instead of polling (ten roles' polls took two thirds of
// the issued instructions, and shared memory's queue from the exponentials).
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool long_wait(uint64_t *bar, uint32_t parity, const DevStatus &st, volatile int *abort_flag,
                                          uint32_t who) {
    if (try_wait_long(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (try_wait_long(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > st.budget_ns) {
            *abort_flag = 1;
            if (st.word) atomicOr(st.word, kStatusTimeout | (who << kStatusWhoShift));
            return false;
        }
    }
}
// The same by a whole warp, whose lanes take the same way out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const DevStatus &st, volatile int *abort_flag,
                                          uint32_t who) {
    return __all_sync(0xffffffffu, long_wait(bar, parity, st, abort_flag, who));
}

// Online log-sum-exp state of one row: M the running maximum (log2 units), l
// the sum of 2^(y - M).  One chunk of W raw logits; hidden ones are -inf.
template <int W>
__device__ __forceinline__ void lse_chunk(const float (&u)[W], float c, float &M, float &l) {
    float m0 = fmaxf(u[0], u[1]), m1 = fmaxf(u[2], u[3]);
#pragma unroll
    for (int k = 4; k < W; k += 4) {
        m0 = fmax3(m0, u[k], u[k + 1]);
        m1 = fmax3(m1, u[k + 2], u[k + 3]);
    }
    const float cm = fmaxf(m0, m1) * c;
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
    for (int k = 0; k < W; k += 2) {
        const int j = (k >> 1) & 1;
        s[j] = f2add(s[j], ex2_pair(f2fma(f2pack(u[k], u[k + 1]), c2, nM)));
    }
    const float2 t = f2unpack(f2add(s[0], s[1]));
    l += t.x + t.y;
}

// Joins a second state of the same row.
__device__ __forceinline__ void lse_join(float &M, float &l, float M1, float l1) {
    const float Mn = fmaxf(M, M1);
    l = (M == -INFINITY ? l : l * ex2(M - Mn)) + (M1 == -INFINITY ? l1 : l1 * ex2(M1 - Mn));
    M = Mn;
}
__device__ __forceinline__ float lse_value(float M, float l) {
    return l == 0.f ? -INFINITY : 0.69314718055994530942f * ((M == -INFINITY ? 0.f : M) + lg2(l));
}

// Sum over W streamed rows of 2^(u c + nb): nb = -lse * log2(e) of each row.
template <int W>
__device__ __forceinline__ float mass_chunk(const float (&u)[W], float c, const float *nb) {
    const uint64_t c2 = f2splat(c);
    uint64_t s[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < W; k += 4) {
        const float4 b = ld_shared_v4(nb + k);
        s[0] = f2add(s[0], ex2_pair(f2fma(f2pack(u[k], u[k + 1]), c2, f2pack(b.x, b.y))));
        s[1] = f2add(s[1], ex2_pair(f2fma(f2pack(u[k + 2], u[k + 3]), c2, f2pack(b.z, b.w))));
    }
    const float2 t = f2unpack(f2add(s[0], s[1]));
    return t.x + t.y;
}

// The owned row `row` of an item: where its result goes (in mass or lse), or
// -1; in kRowLse also its position in its head.
template <int MODE>
__device__ __forceinline__ long long stat_out(const StatParams &p, const StatItem &it, int row, int &i) {
    if (MODE == kKeyMass) {
        i = it.t * 128 + row;
        return i < p.N_K ? ((long long)it.b * p.Hk + it.hk) * p.N_K + i : -1;
    }
    const RowTile rt = row_tile(p, it.hk, it.t);
    const int g = p.pack ? row / p.N_Q : 0;
    i = rt.row0 + row - g * p.N_Q;
    return row < rt.rows ? ((long long)it.b * p.H + rt.head + g) * p.N_Q + i : -1;
}

template <int D, int MODE>
__global__ void __launch_bounds__(StatCfg<D>::THREADS, 1)
    streamkl_stat_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                         const StatParams p) {
    using C = StatCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sA = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sT = sA + 2 * C::TILE_BYTES;

    __shared__ uint64_t bar_afull[2], bar_afree[2], bar_aready[2], bar_aempty[2];   // rows in smem, in tensor memory
    __shared__ uint64_t bar_full[C::NSTAGE], bar_empty[C::NSTAGE];
    __shared__ uint64_t bar_sfull[C::NBUF], bar_sempty[C::NBUF], bar_ifull[C::NSLOT], bar_iempty[C::NSLOT];
    __shared__ uint64_t bar_quiet[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ int rec[5];
    // kKeyMass: a half's rows: -lse * log2(e), the first, and how many there are | chunks with rows to leave out << 8
    __shared__ uint64_t bar_tfull[C::NWG][C::NTABLE], bar_tempty[C::NWG][C::NTABLE];
    __shared__ __align__(16) float table[C::NWG][C::NTABLE][64];
    __shared__ int2 table_rows[C::NWG][C::NTABLE];
    __shared__ float sums[C::NSLOT][C::NWG][MODE == kRowLse ? 2 : 1][C::BM];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int off = p.N_K - p.N_Q;

    grid_release();
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_afull[s], 1);
            mbar_init(&bar_afree[s], 4);
            mbar_init(&bar_aready[s], 4);
            mbar_init(&bar_aempty[s], p.halves);
        }
        for (int s = 0; s < C::NSTAGE; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], p.halves);
        }
        for (int s = 0; s < C::NBUF; ++s) {
            mbar_init(&bar_sfull[s], 1);
            mbar_init(&bar_sempty[s], 4);
        }
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(&bar_ifull[s], 4 * C::NWG);
            mbar_init(&bar_iempty[s], 1);
        }
        for (int s = 0; s < C::NWG * C::NTABLE; ++s) {
            mbar_init(&bar_tfull[0][s], 1);
            mbar_init(&bar_tempty[0][s], 4);
        }
        mbar_init(&bar_quiet[0], 1);
        mbar_init(&bar_quiet[1], 1);
        abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&mQ);
        prefetch_tmap(&mK);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == C::W_EPI) {
        // this CTA's run
        const long long total = stat_total<MODE>(p, blockIdx.x == 0), run = stat_run(total, p.grid);
        const long long u0 = (long long)blockIdx.x * run, left = min(total, u0 + run) - u0;
        int b = 0, hk = 0, t = 0, lo = 0;
        if (left > 0) stat_find<MODE>(p, u0, b, hk, t, lo);
        if (lane == 0) {
            rec[0] = b; rec[1] = hk; rec[2] = t; rec[3] = lo; rec[4] = (int)max(left, 0ll);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    volatile int *abort_v = &abort_flag;
    grid_wait();                                              // kKeyMass after a kRowLse: the log-sum-exps
    StatIter<MODE> iter;
    iter.start(p, rec);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            int n_item = 0, t = 0, a_asked = 0;
            bool ok = true;
            const int q_rows = p.pack ? p.pack * p.N_Q : 128; // of a box
            for (; ok && iter.more(); iter.next(p), ++n_item) {
                const StatItem &it = iter.it;
                const int a = n_item & 1;
                ok = n_item < 2 || long_wait(&bar_afree[a], ((n_item >> 1) - 1) & 1, p.st, abort_v, 1);
                if (!ok) break;
                uint8_t *dst = sA + a * C::TILE_BYTES;
                if (MODE == kKeyMass) {
                    load_tile<D>(dst, &mK, &bar_afull[a], it.t * 128, it.hk, it.b, 128, 0, p.N_K, p.Hk, p.B, p.st.word);
                } else {
                    const RowTile rt = row_tile(p, it.hk, it.t);
                    load_tile<D>(dst, &mQ, &bar_afull[a], rt.row0, rt.head, it.b, q_rows, p.pack, p.N_Q, p.H, p.B,
                                 p.st.word);
                }
                ++a_asked;
                RowCursor cur(p, it, MODE == kKeyMass ? it.lo : 0);
                for (int u = it.lo; u < it.lo + it.n; ++u, ++t) {
                    const int s = t % C::NSTAGE, n = t / C::NSTAGE;
                    ok = n == 0 || long_wait(&bar_empty[s], (n - 1) & 1, p.st, abort_v, 2);
                    if (!ok) break;
                    dst = sT + s * C::TILE_BYTES;
                    if (MODE == kKeyMass) {
                        const RowTile rt = cur.tile(p, it.hk);
                        cur.advance(p, 1);
                        load_tile<D>(dst, &mQ, &bar_full[s], rt.row0, rt.head, it.b, q_rows, p.pack, p.N_Q, p.H, p.B,
                                     p.st.word);
                    } else {
                        load_tile<D>(dst, &mK, &bar_full[s], u * 128, it.hk, it.b, 128, 0, p.N_K, p.Hk, p.B, p.st.word);
                    }
                }
            }
            if (*abort_v) {
                // copies in flight land before the CTA's memory is released
                DevStatus quick = p.st;
                quick.budget_ns = 50000000ull;
                volatile int never = 0;
                for (int s = max(0, t - C::NSTAGE); s < t; ++s)
                    mbar_wait(&bar_full[s % C::NSTAGE], (s / C::NSTAGE) & 1, quick, &never, 2);
                for (int s = max(0, a_asked - 2); s < a_asked; ++s)
                    mbar_wait(&bar_afull[s & 1], (s >> 1) & 1, quick, &never, 1);
            }
        }
    } else if (warp < C::W_EPI) {
        // ------------------------------------------------------------ MMA issuers
        const int half = warp - 1;
        if (half < p.halves && elect_one()) {
            const uint64_t t0 = sw128_desc(smem_u32(sT) + half * 64 * 128, 16, 1024);
            const uint32_t id = p.fp16 ? idesc_fp16(C::BM, 64, 0, 0) : idesc_bf16(C::BM, 64, 0, 0);
            int n_item = 0, s = 0, ps = 0, hb = half, use = 0;
            bool ok = true;
            for (; ok && iter.more(); iter.next(p), ++n_item) {
                const int a = n_item & 1;
                if (!long_wait(&bar_aready[a], (n_item >> 1) & 1, p.st, abort_v, 3)) break;
                const uint32_t ta = tmem + C::TMEM_A + a * (D / 2);
                for (int u = 0; u < iter.it.n; ++u) {
                    ok = (use == 0 || long_wait(&bar_sempty[hb], (use - 1) & 1, p.st, abort_v, 5)) &&
                         long_wait(&bar_full[s], ps, p.st, abort_v, 4);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dt = desc_add(t0, s * C::TILE_BYTES);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16_ts(tmem + hb * 64, ta + kk * 8, desc_add(dt, (kk >> 2) * C::BOX + (kk & 3) * 32), id,
                                    kk > 0);
                    mma_commit(&bar_sfull[hb]);
                    mma_commit(&bar_empty[s]);
                    if (++s == C::NSTAGE) { s = 0; ps ^= 1; }
                    if ((hb += p.halves) >= C::NBUF) { hb -= C::NBUF; ++use; }
                }
                if (ok) mma_commit(&bar_aempty[a]);
            }
            mma_quiesce(&bar_quiet[half], p.st, 9);
        }
    } else if (warp < C::W_LOAD) {
        // ------------------------------------------------------------ owned rows
        const int wg = (warp - C::W_EPI) >> 2, sub = warp & 3, row = sub * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(sub * 32) << 16);
        // halves in turn: half index 2 t + half (or t) of the run goes to warpgroup index mod 4
        const int step = C::NWG / p.halves, phase = wg / p.halves, half = wg % p.halves;
        int n_item = 0, t = 0, e = 0, pe = 0;                 // t: tiles before this item; e, pe: table, its parity
        bool ok = true;
        for (; ok && iter.more(); t += iter.it.n, iter.next(p), ++n_item) {
            const StatItem &it = iter.it;
            int i, lim = 0;                                   // lim: first hidden key (rows past the tile's end see none)
            if (stat_out<MODE>(p, it, row, i) >= 0 && MODE == kRowLse) lim = p.causal ? min(it.nk, i + off + 1) : it.nk;
            // row i sees key j iff i >= j - off: of a head's rows, those from `first` on; `last`: the tile's largest
            const int first = MODE == kKeyMass && p.causal ? i - off : 0;
            const int last = MODE == kKeyMass && p.causal ? it.t * 128 + 127 - off : 0;
            float M = -INFINITY, l = 0.f;
            for (int x = (phase - t) & (step - 1); x < it.n; x += step) {
                const int tt = t + x;
                if (MODE == kKeyMass) ok = warp_wait(&bar_tfull[wg][e], pe, p.st, abort_v, 12);
                const int hc = tt * p.halves + half, buf = hc % C::NBUF;
                const int2 info = MODE == kKeyMass ? table_rows[wg][e] : make_int2(0, 64);
                const float *tab = table[wg][e];
                const int row0 = info.x, chunks = ((info.y & 255) + 31) >> 5;
                ok = ok && warp_wait(&bar_sfull[buf], (hc / C::NBUF) & 1, p.st, abort_v, 6);
                if (!ok) break;
                tc_fence_after();
                const uint32_t logits = lane_base + buf * 64;
                auto release = [&]() {                        // the logits are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_sempty[buf]);
                };
                // two bodies: masks in the common one would cost copies of its registers
                const int c0 = (it.lo + x) * C::BN + half * 64;              // kRowLse: the half's first key
                const bool plain = MODE == kRowLse ? __all_sync(0xffffffffu, c0 + 64 <= lim)
                                                   : chunks == 2 && info.y < 256 && last <= (p.pack ? 0 : row0);
                if (plain) {
                    // 16 columns are loaded while the 16 before them are summed
                    float sum = 0.f, u[2][16];
                    tmem_ld16(logits, u[0]);
#pragma unroll
                    for (int x4 = 0; x4 < 4; ++x4) {
                        tmem_ld_wait_bind(u[x4 & 1]);
                        if (x4 < 3) tmem_ld16(logits + (x4 + 1) * 16, u[(x4 + 1) & 1]);
                        else release();
                        if (MODE == kRowLse) lse_chunk(u[x4 & 1], p.c, M, l);
                        else sum += mass_chunk(u[x4 & 1], p.c, tab + x4 * 16);
                    }
                    l += sum;         // tile by tile: a long sum's rounding grows with its number of terms
                } else {
                    // hidden logits, and those of rows to leave out, become -inf: 2^-inf adds nothing
                    for (int x2 = 0; x2 < chunks; ++x2) {
                        float u[32];
                        tmem_ld32(logits + x2 * 32, u);
                        tmem_ld_wait();
                        const int r0 = row0 + x2 * 32;
                        int h = MODE == kRowLse ? lim - c0 - x2 * 32 : first - r0;   // keys below h are seen; rows from h on see
                        if (MODE == kKeyMass && last <= (p.pack ? 0 : r0)) {
                            // every row sees the keys
                        } else if (MODE == kKeyMass && p.pack) {
                            uint32_t seen = 0u;
                            for (int k = 0; k < 32; ++k)
                                if ((r0 + k) % p.N_Q >= first) seen |= 1u << k;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((seen >> k) & 1u)) u[k] = -INFINITY;
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (MODE == kRowLse ? k >= h : k < h) u[k] = -INFINITY;
                        }
                        if (MODE == kRowLse) {
                            lse_chunk(u, p.c, M, l);
                        } else {
                            if ((info.y >> (8 + x2)) & 1) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if (tab[x2 * 32 + k] == -INFINITY) u[k] = -INFINITY;
                            }
                            l += mass_chunk(u, p.c, tab + x2 * 32);
                        }
                    }
                    release();
                }
                if (MODE == kKeyMass) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_tempty[wg][e]);
                    if (++e == C::NTABLE) { e = 0; pe ^= 1; }
                }
            }
            const int slot = n_item % C::NSLOT, use = n_item / C::NSLOT;
            ok = ok && (use == 0 || warp_wait(&bar_iempty[slot], (use - 1) & 1, p.st, abort_v, 8));
            if (!ok) break;
            sums[slot][wg][0][row] = l;
            if (MODE == kRowLse) sums[slot][wg][1][row] = M;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_ifull[slot]);
        }
    } else if (warp < C::W_OUT) {
        // ------------------------------------------------------------ rows to tensor memory
        const int sub = warp & 3, row = sub * 32 + lane;
        const uint32_t dst = tmem + ((uint32_t)(sub * 32) << 16) + C::TMEM_A;
        // tables for warpgroup `wg`
        const int wg = warp - C::W_LOAD, step = C::NWG / p.halves, phase = wg / p.halves, half = wg % p.halves;
        bool ok = true;
        for (int n_item = 0, t = 0, e = 0, use_e = 0; ok && iter.more(); t += iter.it.n, iter.next(p), ++n_item) {
            const int a = n_item & 1, use = n_item >> 1;
            if (!warp_wait(&bar_afull[a], use & 1, p.st, abort_v, 7)) break;
            if (use > 0 && !warp_wait(&bar_aempty[a], (use - 1) & 1, p.st, abort_v, 11)) break;
            tc_fence_after();
            const uint8_t *src = sA + a * C::TILE_BYTES;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {                // 32 elements, 16 columns
                uint32_t v[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int e = x * 32 + k * 8;
                    const uint4 q = *reinterpret_cast<const uint4 *>(src + (e / 64) * C::BOX + sw128_offset(row, e % 64));
                    v[4 * k] = q.x; v[4 * k + 1] = q.y; v[4 * k + 2] = q.z; v[4 * k + 3] = q.w;
                }
                tmem_st16(dst + a * (D / 2) + x * 16, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar_afree[a]);
                mbar_arrive(&bar_aready[a]);
            }
            if (MODE != kKeyMass) continue;
            const StatItem &it = iter.it;
            const int x0 = (phase - t) & (step - 1);
            RowCursor cur(p, it, it.lo + x0);
            RowTile rt = {0, 0, 0};
            float ahead[2];                                   // log-sum-exps of the half's rows (packed heads follow)
            auto load_lse = [&]() {
                rt = cur.tile(p, it.hk);
                rt.row0 += half * 64;
                rt.rows = max(0, min(rt.rows - half * 64, 64));
                const float *lse = p.lse + ((size_t)it.b * p.H + rt.head) * p.N_Q + rt.row0;
                const bool in = bound_ok(it.b < p.B && rt.head < p.H && rt.row0 >= 0, p.st.word, kSiteConst);
#pragma unroll
                for (int k = 0; k < 2; ++k) ahead[k] = in && k * 32 + lane < rt.rows ? lse[k * 32 + lane] : 0.f;
            };
            if (x0 < it.n) load_lse();
            for (int x = x0; x < it.n; x += step) {
                float nb[2];
                int rows = rt.rows;
                const int row0 = rt.row0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool in = k * 32 + lane < rt.rows, none = fabsf(ahead[k]) == INFINITY;
                    nb[k] = in && !none ? -1.4426950408889634074f * ahead[k] : -INFINITY;
                    // (rows past a head's end are zeros, those past packed heads are not)
                    if (__any_sync(0xffffffffu, in ? none : p.pack > 0)) rows |= 256 << k;
                }
                if (x + step < it.n) {
                    cur.advance(p, step);
                    load_lse();
                }
                ok = use_e == 0 || warp_wait(&bar_tempty[wg][e], (use_e - 1) & 1, p.st, abort_v, 13);
                if (!ok) break;
                table[wg][e][lane] = nb[0];
                table[wg][e][32 + lane] = nb[1];
                if (lane == 0) table_rows[wg][e] = make_int2(row0, rows);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_tfull[wg][e]);
                if (++e == C::NTABLE) { e = 0; ++use_e; }
            }
        }
    } else {
        // ------------------------------------------------------------ writer
        for (int n_item = 0; iter.more(); iter.next(p), ++n_item) {
            const StatItem &it = iter.it;
            const int slot = n_item % C::NSLOT;
            if (!warp_wait(&bar_ifull[slot], (n_item / C::NSLOT) & 1, p.st, abort_v, 10)) break;
            const bool whole = it.n == it.count;
            // an item that two runs share: this run's first item, or its last
            float *part = p.part + ((size_t)blockIdx.x * 2 + (n_item > 0 ? 1 : 0)) * 2 * C::BM;
#pragma unroll
            for (int r = lane; r < C::BM; r += 32) {
                float l = sums[slot][0][0][r], M = MODE == kRowLse ? sums[slot][0][1][r] : 0.f;
#pragma unroll
                for (int w = 1; w < C::NWG; ++w) {
                    if (MODE == kRowLse) lse_join(M, l, sums[slot][w][1][r], sums[slot][w][0][r]);
                    else l += sums[slot][w][0][r];
                }
                int i;
                const long long at = stat_out<MODE>(p, it, r, i);
                if (MODE == kKeyMass && i >= it.nk) l = 0.f;  // keys past the length received nothing
                if (!whole) {
                    part[r] = l;
                    if (MODE == kRowLse) part[C::BM + r] = M;
                } else if (at >= 0 && bound_ok(at < (MODE == kKeyMass ? (long long)p.B * p.Hk * p.N_K
                                                                      : (long long)p.B * p.H * p.N_Q),
                                               p.st.word, kSiteRowOut)) {
                    if (MODE == kRowLse) p.lse[at] = lse_value(M, l);
                    else p.mass[at] = p.accumulate ? p.mass[at] + l : l;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_iempty[slot]);
        }
        // items without a tile (all keys of the batch element, or of the key tile, are padding)
        if (p.kv_len && !(MODE == kKeyMass && p.accumulate)) {
            const int per = MODE == kKeyMass ? (p.N_K + 127) / 128 : p.R * (p.pack ? 1 : p.G);
            for (long long x = blockIdx.x; x < (long long)p.B * p.Hk * per; x += gridDim.x) {
                StatItem it;
                it.t = (int)(x % per);
                it.hk = (int)(x / per % p.Hk);
                it.b = (int)(x / per / p.Hk);
                it.nk = key_count(p.kv_len, it.b, p.N_K, p.st.word, false);
                if (MODE == kKeyMass ? it.t * 128 < it.nk : it.nk > 0) continue;
                for (int r = lane; r < C::BM; r += 32) {
                    int i;
                    const long long at = stat_out<MODE>(p, it, r, i);
                    if (at >= 0) (MODE == kKeyMass ? p.mass : p.lse)[at] = MODE == kKeyMass ? 0.f : -INFINITY;
                }
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

// Joins the partial sums of the items that several runs share: block k the one
// that the end of run k cuts, if it starts in that run.
template <int MODE>
__global__ void __launch_bounds__(128) streamkl_stat_finish_kernel(const StatParams p) {
    __shared__ long long rec[5];
    grid_release();
    if (threadIdx.x < 32) {
        const long long total = stat_total<MODE>(p, false), run = stat_run(total, p.grid);
        const long long u = ((long long)blockIdx.x + 1) * run;
        int b = 0, hk = 0, t = 0, lo = 0;
        if (u < total) stat_find<MODE>(p, u, b, hk, t, lo);
        if (threadIdx.x == 0) {
            rec[0] = b; rec[1] = hk; rec[2] = t;
            rec[3] = lo > 0 && lo <= run ? u - lo : -1;       // the item's first unit
            rec[4] = run;
        }
    }
    __syncthreads();
    grid_wait();
    const long long start = rec[3], run = rec[4];
    if (start < 0) return;
    StatItem it;
    it.b = (int)rec[0]; it.hk = (int)rec[1]; it.t = (int)rec[2];
    it.nk = key_count(p.kv_len, it.b, p.N_K, p.st.word, false);
    const TileList<MODE> l(p, it.nk);
    const long long end = start + l.count(MODE == kKeyMass ? it.t : it.t % l.R);
    const int c0 = (int)(start / run), c1 = (int)((end - 1) / run), r = threadIdx.x;
    float sum = 0.f, M = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
        // it is the first item of a run unless it starts inside
        const float *part = p.part + ((size_t)c * 2 + (c == c0 && start > c * run ? 1 : 0)) * 2 * 128;
        if (MODE == kRowLse) lse_join(M, sum, part[128 + r], part[r]);
        else sum += part[r];
    }
    int i;
    const long long at = stat_out<MODE>(p, it, r, i);
    if (at < 0) return;
    if (MODE == kRowLse) p.lse[at] = lse_value(M, sum);
    else p.mass[at] = p.accumulate ? p.mass[at] + sum : sum;
}

}  // namespace skl
