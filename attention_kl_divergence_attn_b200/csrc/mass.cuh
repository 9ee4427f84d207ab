// mass.cuh — column sums of one softmax matrix: the attention weight that each
// key has received from a set of query rows,
//     lse_i  = log sum_j exp(y_ij),   y_ij = scale q_i . k_j  (visible j)
//     mass_j = sum_{heads of the group} sum_i exp(y_ij - lse_i)
// without writing the matrix.  Both sums run in one kernel template:
//   MODE = kRowLse: an item is 256 query rows, the keys are streamed.
//   MODE = kKeyMass: an item is 256 keys of one key head, the query rows of all
//          heads of its group are streamed.
// The item's rows are the MMA's M dimension (tensor-memory lanes, two MMAs a
// streamed tile), the streamed ones its N dimension, so in both modes a thread
// reads one owned row of a logit tile and its sum over the streamed rows stays
// in the thread.  Up to 64 query rows a head are packed: a tile of 128 rows holds
// as many whole heads as fit.
//
// One CTA an SM.  The tiles of all items are one list, of which every CTA takes
// an equal run, so that causal, padded and few-item problems balance alike; an
// item that two runs share leaves partial sums, which the finish kernel adds in
// a fixed order (the same bits run to run).
//   warp 0      producer: TMA loads of an item's rows and of the streamed tiles
//               (128 rows, a ring).
//   warps 1, 2  MMA issuers, one a half (64 rows) of the streamed tiles.  Warp 1
//               owns the tensor memory: four 128 x 64 logit tiles of fp32 (item
//               half, tile half), and the item's rows (two buffers, packed 16-bit)
//               as the A operand, so that a tcgen05.mma reads only the streamed
//               tile from shared memory (with A in shared memory too, 128 x 128
//               logits took 870 clocks of its bandwidth instead of 512).
//   warps 3..18 four warpgroups, one a logit tile; thread = owned row.
//   warps 19..22 copy an item's rows from shared to tensor memory, an item ahead,
//               and add and write the warpgroups' sums of an item.
//   warp 23     in kKeyMass writes the -lse * log2(e) of a tile's rows as tables for
//               the warpgroups.
// Work bound: one exponential a pair (16 a clock and SM: 2048 clocks a tile)
// against 2 d flops (1024 clocks a tile at d = 128) and 32 KB of streamed rows
// from L2 (items of 128 rows read them twice as often, 9 TB/s over all SMs).
// Measured: 338 us for 8192 causal rows of 32 heads over 8, d = 128, on inputs in
// turn (68 % of the exponentials' rate; 318 us and 73 % on one input again and
// again); 22 us for 2 x 8 heads of 2048 rows, d = 64.
#pragma once

#include "sm100.cuh"

namespace skl {

enum StatMode { kRowLse = 0, kKeyMass = 1 };

constexpr unsigned long long kTileBudgetNs = 20000;   // and a tile that a wait lasts over (some 15 times what one takes)

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
    float *part;                 // [grid][2][2][256]: partial sums of a run's first and last item
    int grid;                    // runs
    DevStatus st;
};

template <int D>
struct StatCfg {
    static constexpr int BM = 256, BN = 128;                  // rows of an item, of a streamed tile
    static constexpr int BOX = 128 * 128;                     // [128 rows][64 columns] 16-bit
    static constexpr int TILE_BYTES = 128 * D * 2;
    static constexpr int NSTAGE = D == 128 ? 4 : 8;
    static constexpr uint32_t TMEM_A = 256;                   // the item's rows: two buffers of two tiles of D / 2 columns
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr int SMEM = (2 + NSTAGE) * TILE_BYTES + 1024;
    static constexpr int NWG = 4;                             // and logit tiles: warpgroup 2 m + h has item half m, tile half h
    static constexpr int W_EPI = 3, W_LOAD = W_EPI + 4 * NWG, W_TABLE = W_LOAD + 4; // first warps of the roles
    static constexpr int NTABLE = 4;                          // tables a tile half
    static constexpr int NSLOT = 4;                           // items whose sums wait for the writer
    static constexpr int THREADS = 32 * (W_TABLE + 1);
    static_assert(TMEM_A + 2 * D <= TMEM_COLS, "logit tiles and the items' rows fit");
};

// ---------------------------------------------------------------- the list of tiles
// Within one (batch, key head): `own` items, item t streaming count(t) tiles.
// With o = ceil((N_K - N_Q) / 128) (no causal mask: beyond every tile), in tiles of 128,
//   kKeyMass: keys 256 t .. are seen by row tiles max(0, 2 t - o) .. R - 1 of each head;
//   kRowLse:  row tiles 2 r, 2 r + 1 see key tiles 0 .. min(A, 2 r + 2 + o) - 1, A those with
//             a key; heads (or groups of packed heads) of one tile are taken in pairs.
template <int MODE>
struct TileList {
    int own, A, o, R, mult;      // R: kKeyMass tiles, kRowLse items a head; mult: heads (or packed groups of heads)
    __device__ __forceinline__ TileList(const StatParams &p, int nk) {
        const bool one = p.pack || p.R == 1;                  // tile a head
        A = (nk + 127) / 128;
        R = p.pack ? 1 : (MODE == kKeyMass ? p.R : (p.R + 1) / 2);
        o = p.causal && !(MODE == kRowLse && one) ? (p.N_K - p.N_Q + 127) / 128 : (1 << 28);
        mult = p.pack ? p.R : p.G;
        own = MODE == kKeyMass ? (nk + 255) / 256 : (one ? (mult + 1) / 2 : mult * R);
    }
    // r: t (kKeyMass), the item of its head (kRowLse)
    __device__ __forceinline__ int count(int r) const {
        return MODE == kKeyMass ? mult * (R - max(0, 2 * r - o)) : min(A, 2 * r + 2 + o);
    }
    __device__ __forceinline__ long long before_row(int r) const {       // tiles of the items before r of a head
        const long long x = min(max((A - o - 1) >> 1, 0), r);
        return x * (x + 1 + o) + (r - x) * A;
    }
    __device__ __forceinline__ long long before(int t) const {           // tiles of the items before t
        if (MODE == kKeyMass) {
            const long long t1 = min(o / 2 + 1, t), x = t - t1;          // from t1 on, 2 t > o
            return ((long long)R * t - x * (t1 + t - 1 - o)) * mult;
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
    __device__ __forceinline__ void start(const StatParams &p, const StatItem &it, int u) {
        first = p.causal && !p.pack ? max(0, 2 * it.t - (p.N_K - p.N_Q + 127) / 128) : 0;
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
                                          int pack, int n_rows, int n_heads, int n_b, uint32_t *word) {
    tma_load_rows(dst, map, bar, row0, head, 0, b, n_rows, n_heads, D / 64, n_b, word);
    if (D > 64 && pack)
        tma_load_rows(dst + StatCfg<D>::BOX, map, bar, row0, head, 1, b, n_rows, n_heads, D / 64, n_b, word);
}

// mbar_wait by a whole warp, whose lanes take the same way out.  (One lane
// waiting for the warp took 50 us more of 320: the exchange costs more than 32
// lanes' waits.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const DevStatus &st, volatile int *abort_flag,
                                          uint32_t who) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort_flag, who));
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

// Half m of an item: its query tile (kRowLse), whether it has rows at all.
__device__ __forceinline__ bool item_rows(const StatParams &p, const StatItem &it, int m, RowTile &rt) {
    if (p.pack || p.R == 1) {
        const int q = 2 * it.t + m;
        if (q >= (p.pack ? p.R : p.G)) return false;
        rt = row_tile(p, it.hk, q);
        return true;
    }
    const int per = (p.R + 1) / 2, g = it.t / per, r = 2 * (it.t - g * per) + m;
    if (r >= p.R) return false;
    rt = row_tile(p, it.hk, g * p.R + r);
    return true;
}

// The owned row `row` of an item: where its result goes (in mass or lse), or
// -1; `i`: the key, or the row of its head.
template <int MODE>
__device__ __forceinline__ long long stat_out(const StatParams &p, const StatItem &it, int row, int &i) {
    if (MODE == kKeyMass) {
        i = it.t * 256 + row;
        return i < p.N_K ? ((long long)it.b * p.Hk + it.hk) * p.N_K + i : -1;
    }
    RowTile rt;
    i = 0;
    if (!item_rows(p, it, row >> 7, rt)) return -1;
    row &= 127;
    const int g = p.pack ? row / p.N_Q : 0;
    i = rt.row0 + row - g * p.N_Q;
    return row < rt.rows ? ((long long)it.b * p.H + rt.head + g) * p.N_Q + i : -1;
}

// Values of the result (sums of keys, log-sum-exps of rows), and of the partial sums.
template <int MODE>
__device__ __forceinline__ long long stat_values(const StatParams &p) {
    return MODE == kKeyMass ? (long long)p.B * p.Hk * p.N_K : (long long)p.B * p.H * p.N_Q;
}
__device__ __forceinline__ long long part_values(const StatParams &p) { return (long long)p.grid * 2 * 2 * 256; }

template <int D, int MODE>
__global__ void __launch_bounds__(StatCfg<D>::THREADS, 1)
    streamkl_stat_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                         const StatParams p) {
    using C = StatCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sA = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sT = sA + 2 * C::TILE_BYTES;

    __shared__ uint64_t bar_afull, bar_afree, bar_aready[2], bar_aempty[2];         // rows in smem, in tensor memory
    __shared__ uint64_t bar_full[C::NSTAGE], bar_empty[C::NSTAGE];
    __shared__ uint64_t bar_sfull[C::NWG], bar_sempty[C::NWG], bar_ifull[C::NSLOT], bar_iempty[C::NSLOT];
    __shared__ uint64_t bar_quiet[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ int rec[5];
    // kKeyMass: a half's rows: -lse * log2(e), the first, and how many there are | chunks with rows to leave out << 8
    __shared__ uint64_t bar_tfull[2][C::NTABLE], bar_tempty[2][C::NTABLE];
    __shared__ __align__(16) float table[2][C::NTABLE][64];
    __shared__ int2 table_rows[2][C::NTABLE];
    __shared__ float sums[C::NSLOT][C::NWG][MODE == kRowLse ? 2 : 1][128];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int off = p.N_K - p.N_Q;

    grid_release();
    if (threadIdx.x == 0) {
        mbar_init(&bar_afull, 1);
        mbar_init(&bar_afree, 4);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_aready[s], 4);
            mbar_init(&bar_aempty[s], p.halves);
        }
        for (int s = 0; s < C::NSTAGE; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], p.halves);
        }
        for (int s = 0; s < C::NWG; ++s) {
            mbar_init(&bar_sfull[s], MODE == kKeyMass ? 2 : 1);     // the MMAs, and the issuer once it has the table
            mbar_init(&bar_sempty[s], 4);
        }
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(&bar_ifull[s], 4 * C::NWG);
            mbar_init(&bar_iempty[s], 4);
        }
        for (int s = 0; s < 2 * C::NTABLE; ++s) {
            mbar_init(&bar_tfull[0][s], 1);
            mbar_init(&bar_tempty[0][s], 8);                  // the warps of both item halves
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
    if (p.pack) {
        // the rows past packed heads, which no copy fills
        for (int x = threadIdx.x; x < (2 + C::NSTAGE) * C::TILE_BYTES / 16; x += C::THREADS)
            reinterpret_cast<uint4 *>(sA)[x] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
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
                ok = n_item == 0 || mbar_wait(&bar_afree, (n_item - 1) & 1, p.st, abort_v, 1);
                if (!ok) break;
                uint8_t *dst = sA;
                RowTile r0 = {0, 0, 0}, r1 = r0;
                const bool two = MODE == kKeyMass ? it.t * 256 + 128 < p.N_K : item_rows(p, it, 1, r1);
                mbar_expect_tx(&bar_afull, (two ? 2 : 1) * (MODE == kKeyMass ? 128 : q_rows) * D * 2);
                if (MODE == kKeyMass) {
                    load_tile<D>(dst, &mK, &bar_afull, it.t * 256, it.hk, it.b, 0, p.N_K, p.Hk, p.B, p.st.word);
                    if (two)
                        load_tile<D>(dst + C::TILE_BYTES, &mK, &bar_afull, it.t * 256 + 128, it.hk, it.b, 0, p.N_K, p.Hk,
                                     p.B, p.st.word);
                } else {
                    item_rows(p, it, 0, r0);
                    load_tile<D>(dst, &mQ, &bar_afull, r0.row0, r0.head, it.b, p.pack, p.N_Q, p.H, p.B, p.st.word);
                    if (two)
                        load_tile<D>(dst + C::TILE_BYTES, &mQ, &bar_afull, r1.row0, r1.head, it.b, p.pack, p.N_Q, p.H,
                                     p.B, p.st.word);
                }
                ++a_asked;
                RowCursor cur = {0, 0, 0};
                if (MODE == kKeyMass) cur.start(p, it, it.lo);
                for (int u = it.lo; u < it.lo + it.n; ++u, ++t) {
                    const int s = t % C::NSTAGE, n = t / C::NSTAGE;
                    ok = n == 0 || mbar_wait(&bar_empty[s], (n - 1) & 1, p.st, abort_v, 2);
                    if (!ok) break;
                    dst = sT + s * C::TILE_BYTES;
                    if (MODE == kKeyMass) {
                        const RowTile rt = cur.tile(p, it.hk);
                        cur.advance(p, 1);
                        mbar_expect_tx(&bar_full[s], q_rows * D * 2);
                        load_tile<D>(dst, &mQ, &bar_full[s], rt.row0, rt.head, it.b, p.pack, p.N_Q, p.H, p.B, p.st.word);
                    } else {
                        mbar_expect_tx(&bar_full[s], 128 * D * 2);
                        load_tile<D>(dst, &mK, &bar_full[s], u * 128, it.hk, it.b, 0, p.N_K, p.Hk, p.B, p.st.word);
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
                if (a_asked > 0) mbar_wait(&bar_afull, (a_asked - 1) & 1, quick, &never, 1);
            }
        }
    } else if (warp < C::W_EPI) {
        // ------------------------------------------------------------ MMA issuers
        const int half = warp - 1;
        if (half < p.halves && elect_one()) {
            const uint64_t t0 = sw128_desc(smem_u32(sT) + half * 64 * 128, 16, 1024);
            const uint32_t id = p.fp16 ? idesc_fp16(128, 64, 0, 0) : idesc_bf16(128, 64, 0, 0);
            int n_item = 0, s = 0, ps = 0, t = 0, e = 0, pe = 0;
            bool ok = true;
            for (; ok && iter.more(); iter.next(p), ++n_item) {
                const int a = n_item & 1;
                if (!mbar_wait(&bar_aready[a], (n_item >> 1) & 1, p.st, abort_v, 3)) break;
                const uint32_t ta = tmem + C::TMEM_A + a * D;
                for (int u = 0; u < iter.it.n; ++u, ++t) {
                    // The issuer waits for the half's table too, and its own arrival hands
                    // the table on: a wait less in each of sixteen warps.
                    ok = (MODE != kKeyMass || mbar_wait(&bar_tfull[half][e], pe, p.st, abort_v, 12)) &&
                         mbar_wait(&bar_full[s], ps, p.st, abort_v, 4);
                    if (!ok) break;
                    const uint64_t dt = desc_add(t0, s * C::TILE_BYTES);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int buf = 2 * m + half;
                        if (!(ok = t == 0 || mbar_wait(&bar_sempty[buf], (t - 1) & 1, p.st, abort_v, 5))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_bf16_ts(tmem + buf * 64, ta + m * (D / 2) + kk * 8,
                                        desc_add(dt, (kk >> 2) * C::BOX + (kk & 3) * 32), id, kk > 0);
                        mma_commit(&bar_sfull[buf]);
                        if (MODE == kKeyMass) mbar_arrive(&bar_sfull[buf]);
                    }
                    if (!ok) break;
                    mma_commit(&bar_empty[s]);
                    if (++s == C::NSTAGE) { s = 0; ps ^= 1; }
                    if (++e == C::NTABLE) { e = 0; pe ^= 1; }
                }
                if (ok) mma_commit(&bar_aempty[a]);
            }
            mma_quiesce(&bar_quiet[half], p.st, 9);
        }
    } else if (warp < C::W_LOAD) {
        // ------------------------------------------------------------ owned rows
        const int wg = (warp - C::W_EPI) >> 2, m = wg >> 1, half = wg & 1, sub = warp & 3;
        const int lrow = sub * 32 + lane, row = m * 128 + lrow;
        const uint32_t logits = tmem + ((uint32_t)(sub * 32) << 16) + wg * 64;
        int n_item = 0, t = 0, e = 0;                         // t: tiles so far; e: table
        bool ok = true;
        for (; ok && iter.more(); iter.next(p), ++n_item) {
            const StatItem &it = iter.it;
            int i;
            const bool mine = stat_out<MODE>(p, it, row, i) >= 0;
            // first hidden key (a row past the tile's end has no say in which body is taken)
            const int lim = MODE == kRowLse && mine && p.causal ? min(it.nk, i + off + 1) : it.nk;
            const bool idle = !__any_sync(0xffffffffu, mine); // nothing of the item is this warp's
            // row i sees key j iff i >= j - off: of a head's rows, those from `first` on; `last`: the tile's largest
            const int first = MODE == kKeyMass && p.causal ? i - off : 0;
            const int last = MODE == kKeyMass && p.causal ? it.t * 256 + m * 128 + 127 - off : 0;
            float M = -INFINITY, l = 0.f;
            for (int x = half < p.halves ? 0 : it.n; x < it.n; ++x, ++t) {
                ok = warp_wait(&bar_sfull[wg], t & 1, p.st, abort_v, 6);
                if (!ok) break;
                const int2 info = MODE == kKeyMass ? table_rows[half][e] : make_int2(0, 64);
                const float *tab = table[half][e];
                const int row0 = info.x, chunks = idle ? 0 : ((info.y & 255) + 31) >> 5;
                tc_fence_after();
                auto release = [&]() {                        // the logits are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_sempty[wg]);
                };
                // two bodies: masks in the common one would cost copies of its registers
                const int c0 = (it.lo + x) * C::BN + half * 64;              // kRowLse: the half's first key
                const bool plain = MODE == kRowLse ? !idle && __all_sync(0xffffffffu, c0 + 64 <= lim)
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
                    bool masks = MODE == kRowLse || last > (p.pack ? 0 : row0);
                    float sum = 0.f;
                    if (!masks) {
                        // Rows to leave out, and zero rows past the tile's end, add 2^-inf; only a key that is
                        // not finite (or such a row) makes that NaN, and the masked sum is taken then.
                        for (int x4 = 0; x4 < 2 * chunks; ++x4) {
                            float u[16];
                            tmem_ld16(logits + x4 * 16, u);
                            tmem_ld_wait();
                            sum += mass_chunk(u, p.c, tab + x4 * 16);
                        }
                        masks = __any_sync(0xffffffffu, sum != sum);
                        if (masks) sum = 0.f;
                    }
                    // hidden logits, and those of rows to leave out, become -inf: 2^-inf adds nothing
                    for (int x2 = masks ? 0 : chunks; x2 < chunks; ++x2) {
                        const int r0 = row0 + x2 * 32, h = MODE == kRowLse ? lim - c0 - x2 * 32 : first - r0;
                        if (MODE == kRowLse ? __all_sync(0xffffffffu, h <= 0) : !p.pack && last - 127 - r0 >= 32)
                            continue;                         // nothing seen
                        float u[32];
                        tmem_ld32(logits + x2 * 32, u);
                        tmem_ld_wait();
                        if (MODE == kRowLse) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (k >= h) u[k] = -INFINITY;
                            lse_chunk(u, p.c, M, l);
                            continue;
                        }
                        if (last > 0 && p.pack) {
                            uint32_t seen = 0u;
                            for (int k = 0; k < 32; ++k)
                                if ((r0 + k) % p.N_Q >= first) seen |= 1u << k;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((seen >> k) & 1u)) u[k] = -INFINITY;
                        } else if (last > r0 && !p.pack) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (k < h) u[k] = -INFINITY;
                        }
                        if ((info.y >> (8 + x2)) & 1) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (tab[x2 * 32 + k] == -INFINITY) u[k] = -INFINITY;
                        }
                        sum += mass_chunk(u, p.c, tab + x2 * 32);
                    }
                    l += sum;
                    release();
                }
                if (MODE == kKeyMass) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_tempty[half][e]);
                    if (++e == C::NTABLE) e = 0;
                }
            }
            const int slot = n_item % C::NSLOT, use = n_item / C::NSLOT;
            ok = ok && (use == 0 || warp_wait(&bar_iempty[slot], (use - 1) & 1, p.st, abort_v, 8));
            if (!ok) break;
            sums[slot][wg][0][lrow] = l;
            if (MODE == kRowLse) sums[slot][wg][1][lrow] = M;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_ifull[slot]);
        }
    } else if (warp < C::W_TABLE) {
        // ------------------------------------------------------------ rows to tensor memory, sums out
        const int sub = warp & 3, row = sub * 32 + lane;
        const uint32_t dst = tmem + ((uint32_t)(sub * 32) << 16) + C::TMEM_A;
        // Two waits last as long as an item: for the next item's rows, which are asked for behind
        // its last tile, and for its sums.  An item may have millions of tiles of one to three
        // microseconds, so those waits' limit grows with it (the other roles' stays, and ends these too).
        auto patient = [&](int tiles) -> DevStatus {
            DevStatus st = p.st;
            st.budget_ns += (unsigned long long)tiles * kTileBudgetNs;
            return st;
        };
        auto copy = [&](int n_item, int tiles) -> bool {      // `tiles`: of the item before it
            const int a = n_item & 1, use = n_item >> 1;
            if (!warp_wait(&bar_afull, n_item & 1, patient(tiles), abort_v, 7)) return false;
            if (use > 0 && !warp_wait(&bar_aempty[a], (use - 1) & 1, p.st, abort_v, 11)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < 2; ++m) {
                const uint8_t *src = sA + m * C::TILE_BYTES;
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {            // 32 elements, 16 columns
                    uint32_t v[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = x * 32 + k * 8;
                        const uint4 q =
                            *reinterpret_cast<const uint4 *>(src + (c / 64) * C::BOX + sw128_offset(row, c % 64));
                        v[4 * k] = q.x; v[4 * k + 1] = q.y; v[4 * k + 2] = q.z; v[4 * k + 3] = q.w;
                    }
                    tmem_st16(dst + a * D + m * (D / 2) + x * 16, v);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar_afree);
                mbar_arrive(&bar_aready[a]);
            }
            return true;
        };
        // this warp's 64 rows of an item: the sums of two warpgroups
        auto write = [&](const StatItem &it, int n_item) -> bool {
            const int slot = n_item % C::NSLOT;
            if (!warp_wait(&bar_ifull[slot], (n_item / C::NSLOT) & 1, patient(it.n), abort_v, 10)) return false;
            const bool whole = it.n == it.count;
            // an item that two runs share: this run's first item, or its last
            float *part = p.part + ((size_t)blockIdx.x * 2 + (n_item > 0 ? 1 : 0)) * 2 * C::BM;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int w = 2 * k, q = row, r = k * 128 + row;
                float l = sums[slot][w][0][q], M = MODE == kRowLse ? sums[slot][w][1][q] : 0.f;
                if (MODE == kRowLse) lse_join(M, l, sums[slot][w + 1][1][q], sums[slot][w + 1][0][q]);
                else l += sums[slot][w + 1][0][q];
                int i;
                const long long at = stat_out<MODE>(p, it, r, i);
                if (MODE == kKeyMass && i >= it.nk) l = 0.f;  // keys past the length received nothing
                if (!whole) {
                    if (!bound_ok(part + C::BM + r < p.part + part_values(p), p.st.word, kSitePart)) continue;
                    part[r] = l;
                    if (MODE == kRowLse) part[C::BM + r] = M;
                } else if (at >= 0 && bound_ok(at < stat_values<MODE>(p), p.st.word, kSiteRowOut)) {
                    if (MODE == kRowLse) p.lse[at] = lse_value(M, l);
                    else p.mass[at] = p.accumulate ? p.mass[at] + l : l;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_iempty[slot]);
            return true;
        };
        bool ok = !iter.more() || copy(0, 0);
        for (int n_item = 0; ok && iter.more(); ++n_item) {
            const StatItem it = iter.it;
            iter.next(p);
            ok = (!iter.more() || copy(n_item + 1, it.n)) && write(it, n_item);
        }
    } else if (MODE == kKeyMass) {
        // ------------------------------------------------------------ tables
        int e = 0, use_e = 0, x = 0;
        float l[4];                                           // log-sum-exps of a tile's rows (packed heads follow)
        RowTile rt = {0, 0, 0};
        auto load_lse = [&](const RowCursor &cur) {
            rt = cur.tile(p, iter.it.hk);
            const long long first = ((long long)iter.it.b * p.H + rt.head) * p.N_Q + rt.row0;
            const float *lse = p.lse + first;
            const bool in = bound_ok(iter.it.b < p.B && rt.head < p.H && rt.row0 >= 0 &&
                                         first + rt.rows <= (long long)p.B * p.H * p.N_Q,
                                     p.st.word, kSiteConst);
#pragma unroll
            for (int k = 0; k < 4; ++k) l[k] = in && k * 32 + lane < rt.rows ? lse[k * 32 + lane] : 0.f;
        };
        RowCursor cur = {0, 0, 0};
        bool more = iter.more();
        if (more) {
            cur.start(p, iter.it, iter.it.lo);
            load_lse(cur);
        }
        while (more) {
            float nb[4];
            uint32_t odd = 0u;
            const int row0 = rt.row0, rows = rt.rows;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = k * 32 + lane < rows, none = fabsf(l[k]) == INFINITY;
                nb[k] = in && !none ? -1.4426950408889634074f * l[k] : -INFINITY;
                if (__any_sync(0xffffffffu, !in || none)) odd |= 1u << k;
            }
            // the next tile's are loaded while this one's wait for their place
            if (++x < iter.it.n) {
                cur.advance(p, 1);
            } else {
                x = 0;
                iter.next(p);
                if ((more = iter.more())) cur.start(p, iter.it, iter.it.lo);
            }
            if (more) load_lse(cur);
            for (int h = 0; h < p.halves; ++h) {
                if (use_e > 0 && !warp_wait(&bar_tempty[h][e], (use_e - 1) & 1, p.st, abort_v, 13)) {
                    more = false;
                    break;
                }
                table[h][e][lane] = h ? nb[2] : nb[0];
                table[h][e][32 + lane] = h ? nb[3] : nb[1];
                if (lane == 0)
                    table_rows[h][e] =
                        make_int2(row0 + h * 64, max(0, min(rows - h * 64, 64)) | ((odd >> (2 * h)) & 3u) << 8);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_tfull[h][e]);
            }
            if (++e == C::NTABLE) { e = 0; ++use_e; }
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
__global__ void __launch_bounds__(256) streamkl_stat_finish_kernel(const StatParams p) {
    __shared__ long long rec[5];
    grid_release();
    if (threadIdx.x < 32) {
        const long long total = stat_total<MODE>(p, false), run = stat_run(total, p.grid);
        const long long u = ((long long)blockIdx.x + 1) * run;
        int b = 0, hk = 0, t = 0, lo = 0;
        if (u < total && (int)blockIdx.x + 1 < p.grid) stat_find<MODE>(p, u, b, hk, t, lo);
        if (threadIdx.x == 0) {
            rec[0] = b; rec[1] = hk; rec[2] = t;
            rec[3] = lo > 0 && lo <= run ? u - lo : -1;       // the item's first unit
            rec[4] = run;
        }
    }
    // Items without a tile (all keys of the batch element, or of the key tile, are
    // padding): written by nobody else, so at once.
    if (p.kv_len && !(MODE == kKeyMass && p.accumulate)) {
        const int per = MODE == kKeyMass ? (p.N_K + 255) / 256 : TileList<MODE>(p, p.N_K).own;
        for (long long x = blockIdx.x; x < (long long)p.B * p.Hk * per; x += gridDim.x) {
            StatItem it;
            it.t = (int)(x % per);
            it.hk = (int)(x / per % p.Hk);
            it.b = (int)(x / per / p.Hk);
            it.nk = key_count(p.kv_len, it.b, p.N_K, p.st.word, false);
            if (MODE == kKeyMass ? it.t * 256 < it.nk : it.nk > 0) continue;
            int i;
            const long long at = stat_out<MODE>(p, it, threadIdx.x, i);
            if (at >= 0 && bound_ok(at < stat_values<MODE>(p), p.st.word, kSiteZero))
                (MODE == kKeyMass ? p.mass : p.lse)[at] = MODE == kKeyMass ? 0.f : -INFINITY;
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
        const float *part = p.part + ((size_t)c * 2 + (c == c0 && start > c * run ? 1 : 0)) * 2 * 256;
        if (!bound_ok(c >= 0 && part + 256 + r < p.part + part_values(p), p.st.word, kSitePart)) continue;
        if (MODE == kRowLse) lse_join(M, sum, part[256 + r], part[r]);
        else sum += part[r];
    }
    int i;
    const long long at = stat_out<MODE>(p, it, r, i);
    if (at < 0 || !bound_ok(at < stat_values<MODE>(p), p.st.word, kSiteRowOut)) return;
    if (MODE == kRowLse) p.lse[at] = lse_value(M, sum);
    else p.mass[at] = p.accumulate ? p.mass[at] + sum : sum;
}

}  // namespace skl
