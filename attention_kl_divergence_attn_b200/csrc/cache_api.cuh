// cache_api.cuh — C entry points of the cache operators (streamkl_key_mass,
// streamkl_decode, streamkl_evict): argument checks and launches.  Included at
// the end of streamkl.cu, whose helpers it uses.
#pragma once

namespace {

enum { kDtypeBf16 = 0, kDtypeFp16 = 1 };
constexpr long long kMaxStride = 1ll << 38;          // elements: 2^39 bytes, inside what a tensor map addresses
constexpr int kMaxCap = 1 << 30;                     // slots of a sequence

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A stride triple of a 16-bit tensor whose last dimension is contiguous: rows
// start on 16-byte boundaries.  Dimensions of one element may have any stride.
bool stride_ok(const long long *s, const long long *extent) {
    for (int x = 0; x < 3; ++x) {
        if (extent[x] <= 1) continue;
        if (s[x] <= 0 || s[x] % 8 != 0 || s[x] > kMaxStride) return false;
    }
    return true;
}

// The bytes from a tensor's first element to its last.
struct Span {
    uintptr_t a, z;
};
Span span_of(const void *p, unsigned __int128 bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!p || bytes == 0) return {0, 0};
    return {a, bytes > UINTPTR_MAX - a ? UINTPTR_MAX : a + (uintptr_t)bytes};
}
// 16-bit rows of d elements.  (Of a cache's pages: as many slots as a sequence may reach,
// for a page may be declared larger than that, and than its memory.)
Span rows_span(const void *p, const long long *s, const long long *extent, int d) {
    unsigned __int128 n = d;
    for (int x = 0; x < 3; ++x) {
        if (extent[x] <= 0) return {0, 0};
        if (extent[x] > 1) n += (unsigned __int128)(extent[x] - 1) * (unsigned long long)s[x];
    }
    return span_of(p, 2 * n);
}
Span vec_span(const void *p, long long n) { return span_of(p, 4 * (unsigned __int128)n); }

// Some output overlaps an input or another output.
bool overlapping(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    auto meet = [](const Span &x, const Span &y) { return x.a < y.z && y.a < x.z; };
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (meet(*o, i)) return true;
        for (const Span *q = outs.begin(); q != o; ++q)
            if (meet(*o, *q)) return true;
    }
    return false;
}

// 5-D map over rows of d elements in [n3][n2][n1][d] with strides (in
// elements) s[0], s[1], s[2], as [n3][d / 64][n2][n1][64]: box of `rows` rows x
// `heads` x `blocks` of 64 columns, 128-byte swizzle, zeros outside, so ragged
// tiles read zeros.
bool make_rows_map(CUtensorMap *m, const void *ptr, int d, int n1, int n2, int n3, const long long *s, int rows,
                   int heads, int blocks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t any = (cuuint64_t)d * 2;        // stride of a dimension with one element
    cuuint64_t dims[5] = {64, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)(d / 64), (cuuint64_t)n3};
    cuuint64_t strides[4] = {n1 > 1 ? (cuuint64_t)s[2] * 2 : any, n2 > 1 ? (cuuint64_t)s[1] * 2 : any, 128,
                             n3 > 1 ? (cuuint64_t)s[0] * 2 : any};
    cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)heads, (cuuint32_t)blocks, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query tiles of 128 rows: whole heads of up to 64 rows are packed.
void stat_rows(StatParams *p) {
    p->pack = p->N_Q <= 64 ? std::min(p->G, 128 / p->N_Q) : 0;
    p->R = p->pack ? (p->G + p->pack - 1) / p->pack : (p->N_Q + 127) / 128;
}

// Runs of a call, and scratch for every run's two partial items.
int stat_grid() { return std::max(1, sm_count()); }
size_t stat_bytes() { return (size_t)stat_grid() * 2 * 2 * 256 * sizeof(float); }

bool stat_shape_ok(int B, int H, int H_k, int N_Q, int N_K, int d, int dtype, int causal) {
    if (B < 0 || H < 0 || N_Q < 0 || N_K < 0 || H_k < 1 || (H > 0 && H % H_k != 0)) return false;
    if (causal != 0 && causal != 1) return false;
    if (causal && N_Q > N_K) return false;
    if (!causal && N_K == 0 && N_Q > 0 && B > 0 && H > 0) return false;
    if (dtype != kDtypeBf16 && dtype != kDtypeFp16) return false;
    return (long long)B * H <= (1ll << 24) && (long long)B * H_k <= (1ll << 24) && N_Q <= (1 << 24) && N_K <= (1 << 24) &&
           (long long)H * N_Q < (1ll << 31) &&
           (double)B * H * ((N_Q + 127) / 128) * ((N_K + 127) / 128) < 1e11;      // a run's tiles are counted in 32 bits
}

// scale log2(e), with what the tensor cores leave of an fp16 logit put back.  They round the
// running sum towards zero at each of its d / 16 additions, by half a step on average, which
// is 0.36 2^-23 of it (the mean of step / value over a binade is 0.72 2^-23); of a sum that
// grows evenly that comes to (d / 16 + 1) / 2 times as much.  Measured: large logits came out
// 1.1e-7 (d = 64) and 1.5e-7 to 1.8e-7 (d = 128) too small, and with log-sum-exps from
// elsewhere the sums' error against 64 bits was up to 7 times that of 32-bit torch (1.2e-6
// for 1.6e-7, 1.8e-6 at most in 70 draws); with this it is 0.4 to 3 times, 1.0e-6 at most.
// bf16 products have fewer bits to lose (0.7e-7 and 0.8e-7) and stay as they are, because
// streamkl_fwd's log-sum-exps are off alike, so that it cancels in a weight (an error of
// 4.6e-7 as it is, 1.3e-6 corrected).
float fp16_scale(float scale, int d) {
    return (float)((double)scale * 1.4426950408889634 * (1.0 + 0.36 * (d / 16 + 1) / 2 * 0x1p-23));
}

// Launch with the attributes of a dependent kernel (it may start while its
// predecessor runs and calls grid_wait) and of a cluster, where asked for.
template <typename K, typename... A>
streamkl_status launch_ex(K kern, long long grid, int threads, int smem, cudaStream_t s, bool dependent, int cluster,
                          A... args) {
    cudaLaunchConfig_t c;
    memset(&c, 0, sizeof c);
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = (size_t)smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    if (dependent) {
        at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[c.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[c.numAttrs].val.clusterDim.x = (unsigned)cluster;
        at[c.numAttrs].val.clusterDim.y = 1;
        at[c.numAttrs++].val.clusterDim.z = 1;
    }
    c.attrs = at;
    if (cudaLaunchKernelEx(&c, kern, args...) == cudaSuccess) return STREAMKL_OK;
    (void)cudaGetLastError();                        // reported here
    return STREAMKL_ERR_CUDA;
}

template <int D, int MODE>
streamkl_status launch_stat(const void *q, const long long *qs, const void *k, const long long *ks, StatParams p,
                            bool dependent, cudaStream_t s) {
    using C = StatCfg<D>;
    stat_rows(&p);
    p.halves = MODE == kKeyMass && (p.pack ? p.pack : 1) * p.N_Q <= 64 ? 1 : 2;
    CUtensorMap mq, mk;
    if (!make_rows_map(&mq, q, D, p.N_Q, p.H, p.B, qs, p.pack ? p.N_Q : 128, std::max(1, p.pack),
                       p.pack ? 1 : D / 64) ||
        !make_rows_map(&mk, k, D, p.N_K, p.Hk, p.B, ks, 128, 1, D / 64))
        return STREAMKL_ERR_CUDA;
    // (no more runs than tiles)
    const double tiles = (double)p.B * p.Hk * (p.pack ? p.R : (double)p.G * p.R) * ((p.N_K + 127) / 128);
    p.grid = (int)std::min<double>(stat_grid(), tiles);
    auto kern = streamkl_stat_kernel<D, MODE>;
    if (set_smem(kern, C::SMEM) != cudaSuccess) return STREAMKL_ERR_CUDA;
    streamkl_status st = launch_ex(kern, p.grid, C::THREADS, C::SMEM, s, dependent, 1, mq, mk, p);
    if (st != STREAMKL_OK || (p.grid == 1 && !p.kv_len)) return st;
    return launch_ex(streamkl_stat_finish_kernel<MODE>, std::max(1, p.grid - 1), 256, 0, s, true, 1, p);
}

bool paged_shape_ok(int B, int H, int H_k, int num_pages, int page_size, int max_pages, int dtype) {
    if (B < 0 || H < 0 || H_k < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return false;
    if (H > 0 && H % H_k != 0) return false;
    if (dtype != kDtypeBf16 && dtype != kDtypeFp16) return false;
    return (long long)B * H <= (1ll << 24) && (long long)B * H_k <= (1ll << 24) && B < (1 << 24);
}

bool cache_pointers_ok(const void *k, const void *v, int num_pages, const int *table, int max_pages, const int *len) {
    if (num_pages > 0 && max_pages > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return false;
    return (max_pages == 0 || table) && aligned4(table) && aligned4(len);
}

Span table_span(const int *table, int B, int max_pages, long long stride) {
    return span_of(table, max_pages > 0 ? 4 * ((unsigned __int128)(B - 1) * (unsigned long long)std::max(0ll, stride) +
                                               max_pages) : 0);
}

int paged_cap(int page_size, int max_pages, const void *mass, int mass_cap) {
    long long cap = std::min<long long>((long long)page_size * max_pages, kMaxCap);
    if (mass) cap = std::min<long long>(cap, mass_cap);
    return (int)cap;
}

struct DecodeScratch {
    int grid;
    bool by_row;
    size_t o, ml, logits, total;     // byte offsets and the whole
};

// Sequences of at most this many slots are not split: a CTA streams a whole
// row, and there is no second kernel.  GPU time so / split, us, d = 128, 4 heads
// over each key head, no weights, by slots and rows (sequences x key heads):
//            1 row      8         64          256         1024
//     128    5.3/6.9    5.3/8.7   5.4/9.0     6.7/8.2     22.3/25.8
//     256    7.5/7.5    7.5/8.3   7.6/10.0    9.0/10.5    35.2/37.5
//     512    10.6/7.7   10.6/8.4  10.8/11.4   13.5/19.0   54.1/54.7
//    1024    17.1/8.4   17.1/9.0  17.2/13.7   24.6/30.1   92.8/89.2
// (with weights the rows' sums cost more than a second kernel from 1024 rows of 256
// slots on: 44.0/42.9, and 72.9/62.2 at 512).  The room is known on the host and rows
// are mostly shorter, which is what the bound leans to; a launch saved is 4 us of a
// call's host time besides.
constexpr int kByRowCap = 512;

DecodeScratch decode_scratch(int B, int H, int H_k, int page_size, int max_pages, int d, bool with_mass, int mass_cap) {
    DecodeScratch r;
    const int G = H_k > 0 ? H / H_k : 0, nhb = (G + 15) / 16;
    const int cap = paged_cap(page_size, max_pages, with_mass ? &r : nullptr, mass_cap);
    const long long rows = (long long)B * H_k * nhb, tiles = rows * (((long long)cap + kDecTile - 1) / kDecTile);
    r.by_row = cap <= kByRowCap;
    r.grid = (int)(r.by_row ? rows : std::max<long long>(1, std::min<long long>(2ll * std::max(1, sm_count()), tiles)));
    const size_t parts = r.by_row ? 0 : (size_t)r.grid * 2 * 16;
    r.o = 0;
    r.ml = r.o + parts * d * sizeof(float);
    r.logits = r.ml + parts * 2 * sizeof(float);
    r.total = r.logits + (with_mass ? (size_t)B * H * cap * sizeof(float) : 0);
    return r;
}

// The split kernel counts a call's tiles in 32 bits, the mass blocks of the
// finish kernel are a grid.
bool decode_units_ok(int B, int H, int H_k, int cap, int mass_cap) {
    const long long rows = (long long)B * H_k * ((H / H_k + 15) / 16);
    return rows * ((cap + kDecTile - 1) / kDecTile + 4ll) <= (1ll << 30) &&
           rows * (mass_cap / kFinishTokens + 1ll) <= (1ll << 30);
}

template <typename T, int D>
streamkl_status launch_decode(const DecodeParams &p, cudaStream_t s) {
    auto kern = p.by_row ? streamkl_decode_kernel<T, D, true> : streamkl_decode_kernel<T, D, false>;
    if (set_smem(kern, DecCfg<D>::SMEM) != cudaSuccess) return STREAMKL_ERR_CUDA;
    streamkl_status st = launch_ex(kern, p.grid, kDecWarps * 32, DecCfg<D>::SMEM, s, false, 1, p);
    // (by the weights, not by the saved logits: without room for a slot there are none, and weights to copy still)
    const bool mass = p.mass && p.mass_cap > 0 && !(p.by_row && p.nhb == 1);
    if (st != STREAMKL_OK || (p.by_row && !mass)) return st;
    const long long n_join = p.by_row ? 0 : ((long long)p.B * p.H + 3) / 4;
    const int nx = std::max(1, (p.mass_cap + kFinishTokens - 1) / kFinishTokens);
    const long long n_mass = mass ? (long long)nx * p.B * p.Hk : 0;
    return launch_ex(streamkl_decode_finish_kernel<T, D>, n_join + n_mass, 128, 0, s, true, 1, p, (int)n_join, nx);
}

// Entries of a table up to which each sequence looks for its pages in the
// others' rows, instead of a kernel in which pages are claimed.  GPU time so / with
// claims, us: 65 entries 10.2/10.4, 260 11.0/11.0, 520 11.8/11.5, 1040 (4 sequences)
// 14.1/13.3 or (16) 13.3/12.3, 2080 18.6/16.4 or 14.7/13.0.  The launch saved is 2 us
// of a call's host time (65 entries: 22.0 us a call for 24.1), which is what a call
// takes where this GPU time is less: up to about 1000 entries.
constexpr int kEvictTable = 1024;

struct EvictScratch {
    size_t owner, refused, moves, lists, total;
    int list;
};

EvictScratch evict_scratch(int B, int H_k, int num_pages, int page_size, int max_pages, int mass_cap, int budget) {
    EvictScratch r;
    const int cap = paged_cap(page_size, max_pages, &r, mass_cap);
    r.list = std::min(std::max(budget, 0), std::max(0, cap - std::max(budget, 0)));   // most rows that can move
    r.owner = 0;
    r.refused = r.owner + (size_t)num_pages * sizeof(int);
    r.moves = r.refused + (size_t)B * sizeof(int);
    r.lists = r.moves + (size_t)B * H_k * sizeof(int);
    r.total = r.lists + (size_t)B * H_k * 4 * r.list * sizeof(int);
    return r;
}

}  // namespace

extern "C" {

size_t streamkl_key_mass_scratch_size(int B, int H, int H_k, int N_Q, int N_K, int d, int lse_given) {
    (void)d;
    (void)lse_given;
    if (B <= 0 || H <= 0 || H_k < 1 || H % H_k != 0 || N_Q <= 0 || N_K <= 0) return 0;
    return stat_bytes();
}

streamkl_status streamkl_key_mass(const void *q, const long long *q_stride, const void *k, const long long *k_stride,
                                  int dtype, int B, int H, int H_k, int N_Q, int N_K, int d, float scale, int causal,
                                  const int *kv_len, float *lse, int lse_given, float *mass, int accumulate,
                                  void *workspace, size_t workspace_bytes, void *scratch, size_t scratch_bytes,
                                  void *stream) {
    if (!stat_shape_ok(B, H, H_k, N_Q, N_K, d, dtype, causal)) return STREAMKL_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale == INFINITY) return STREAMKL_ERR_INVALID_ARG;
    if ((lse_given != 0 && lse_given != 1) || (accumulate != 0 && accumulate != 1)) return STREAMKL_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kWorkspaceBytes) return STREAMKL_ERR_WORKSPACE;
    if (!aligned16(workspace) || !aligned16(scratch)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned4(kv_len)) return STREAMKL_ERR_INVALID_ARG;
    const long long n_keys = (long long)B * H_k * N_K, n_rows = (long long)B * H * N_Q;
    if (n_keys > 0 && !mass) return STREAMKL_ERR_INVALID_ARG;
    if (n_keys == 0) return STREAMKL_OK;                     // no keys, so no rows either
    cudaStream_t s = (cudaStream_t)stream;
    if (n_rows == 0) {                                       // nothing looks at the keys
        if (accumulate) return STREAMKL_OK;
        return cudaMemsetAsync(mass, 0, (size_t)n_keys * sizeof(float), s) == cudaSuccess ? STREAMKL_OK
                                                                                         : STREAMKL_ERR_CUDA;
    }
    if (!q || !k || !lse || !aligned16(q) || !aligned16(k)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned4(lse) || !aligned4(mass)) return STREAMKL_ERR_INVALID_ARG;
    const long long qs[3] = {q_stride ? q_stride[0] : (long long)H * N_Q * d, q_stride ? q_stride[1] : (long long)N_Q * d,
                             q_stride ? q_stride[2] : d};
    const long long ks[3] = {k_stride ? k_stride[0] : (long long)H_k * N_K * d,
                             k_stride ? k_stride[1] : (long long)N_K * d, k_stride ? k_stride[2] : d};
    const long long qe[3] = {B, H, N_Q}, ke[3] = {B, H_k, N_K};
    if (!stride_ok(qs, qe) || !stride_ok(ks, ke)) return STREAMKL_ERR_INVALID_ARG;
    if (!scratch || scratch_bytes < stat_bytes()) return STREAMKL_ERR_WORKSPACE;
    const Span lse_span = vec_span(lse, n_rows), none = {0, 0};
    if (overlapping({vec_span(mass, n_keys), lse_given ? none : lse_span},
                    {rows_span(q, qs, qe, d), rows_span(k, ks, ke, d), vec_span(kv_len, B), lse_given ? lse_span : none}))
        return STREAMKL_ERR_INVALID_ARG;
    streamkl_status st = check_device();
    if (st != STREAMKL_OK) return st;

    StatParams p;
    memset(&p, 0, sizeof p);
    p.B = B; p.H = H; p.Hk = H_k; p.G = H / H_k; p.N_Q = N_Q; p.N_K = N_K; p.causal = causal;
    p.kv_len = kv_len;
    p.fp16 = dtype == kDtypeFp16;
    p.c = p.fp16 ? fp16_scale(scale, d) : scale * kLog2e;
    p.lse = lse; p.mass = mass; p.accumulate = accumulate;
    p.part = static_cast<float *>(scratch);
    p.st.word = static_cast<uint32_t *>(workspace);
    p.st.budget_ns = kWaitBudgetNs;
    if (!lse_given) {
        st = d == 64 ? launch_stat<64, kRowLse>(q, qs, k, ks, p, false, s) : launch_stat<128, kRowLse>(q, qs, k, ks, p, false, s);
        if (st != STREAMKL_OK) return st;
    }
    return d == 64 ? launch_stat<64, kKeyMass>(q, qs, k, ks, p, !lse_given, s)
                   : launch_stat<128, kKeyMass>(q, qs, k, ks, p, !lse_given, s);
}

size_t streamkl_decode_scratch_size(int B, int H, int H_k, int page_size, int max_pages, int d, int with_mass,
                                    int mass_cap) {
    if (B <= 0 || H <= 0 || H_k < 1 || H % H_k != 0 || page_size < 1 || max_pages < 0 || d < 1 || mass_cap < 0) return 0;
    return decode_scratch(B, H, H_k, page_size, max_pages, d, with_mass != 0, mass_cap).total;
}

streamkl_status streamkl_decode(const void *q, const long long *q_stride, const void *k_pages,
                                const long long *k_stride, const void *v_pages, const long long *v_stride, int dtype,
                                int B, int H, int H_k, int d, int num_pages, int page_size, const int *page_table,
                                int max_pages, long long table_stride, const int *seq_len, float scale, void *out,
                                float *lse, const float *mass, float *mass_out, int mass_cap, void *workspace,
                                size_t workspace_bytes, void *scratch, size_t scratch_bytes, void *stream) {
    if (!paged_shape_ok(B, H, H_k, num_pages, page_size, max_pages, dtype)) return STREAMKL_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale == INFINITY || mass_cap < 0 || mass_cap > kMaxCap) return STREAMKL_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kWorkspaceBytes) return STREAMKL_ERR_WORKSPACE;
    if (!aligned16(workspace) || !aligned16(scratch)) return STREAMKL_ERR_INVALID_ARG;
    if ((mass == nullptr) != (mass_out == nullptr)) return STREAMKL_ERR_INVALID_ARG;
    if ((long long)B * H == 0) {                             // nothing looks at the keys
        if (B == 0 || mass == mass_out || mass_cap == 0) return STREAMKL_OK;
        return cudaMemcpyAsync(mass_out, mass, (size_t)B * H_k * mass_cap * sizeof(float), cudaMemcpyDeviceToDevice,
                               (cudaStream_t)stream) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
    }
    if (!q || !seq_len || !out || !lse || !aligned16(q) || !aligned16(out)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned4(lse) || !aligned4(mass) || !aligned4(mass_out)) return STREAMKL_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_pages, v_pages, num_pages, page_table, max_pages, seq_len)) return STREAMKL_ERR_INVALID_ARG;
    if (!decode_units_ok(B, H, H_k, paged_cap(page_size, max_pages, mass, mass_cap), mass ? mass_cap : 0))
        return STREAMKL_ERR_INVALID_ARG;
    const DecodeScratch ds = decode_scratch(B, H, H_k, page_size, max_pages, d, mass != nullptr, mass_cap);
    if (ds.total > 0 && (!scratch || scratch_bytes < ds.total)) return STREAMKL_ERR_WORKSPACE;
    const long long qs[3] = {0, q_stride ? q_stride[0] : (long long)H * d, q_stride ? q_stride[1] : d};
    const long long cont[3] = {(long long)H_k * page_size * d, (long long)page_size * d, d};
    const long long *ks = k_stride ? k_stride : cont, *vs = v_stride ? v_stride : cont;
    const long long qe[3] = {1, B, H}, pe[3] = {num_pages, H_k, page_size};
    if (!stride_ok(qs, qe) || !stride_ok(ks, pe) || !stride_ok(vs, pe)) return STREAMKL_ERR_INVALID_ARG;
    if (B > 1 && table_stride < 0) return STREAMKL_ERR_INVALID_ARG;
    const long long rows = (long long)B * H, weights = (long long)B * H_k * mass_cap;
    const long long used[3] = {num_pages, H_k, std::min(page_size, paged_cap(page_size, max_pages, mass, mass_cap))};
    if (overlapping({span_of(out, (unsigned __int128)rows * d * 2), vec_span(lse, rows), vec_span(mass_out, weights)},
                    {rows_span(q, qs, qe, d), rows_span(k_pages, ks, used, d), rows_span(v_pages, vs, used, d),
                     table_span(page_table, B, max_pages, table_stride), vec_span(seq_len, B),
                     vec_span(mass == mass_out ? nullptr : mass, weights)}))
        return STREAMKL_ERR_INVALID_ARG;
    streamkl_status st = check_device();
    if (st != STREAMKL_OK) return st;

    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.B = B; p.H = H; p.Hk = H_k; p.G = H / H_k; p.nhb = (p.G + 15) / 16;
    p.pages = num_pages; p.page = page_size; p.max_pages = max_pages;
    p.cap = paged_cap(page_size, max_pages, mass, mass_cap);
    p.q = q; p.q_b = qs[1]; p.q_h = qs[2];
    p.k = PageView{k_pages, ks[0], ks[1], ks[2]};
    p.v = PageView{v_pages, vs[0], vs[1], vs[2]};
    p.table = page_table; p.table_b = table_stride; p.len = seq_len;
    p.c = scale * kLog2e;
    p.o = out; p.lse = lse;
    char *sc = static_cast<char *>(scratch);
    p.part_o = reinterpret_cast<float *>(sc + ds.o);
    p.part_ml = reinterpret_cast<float *>(sc + ds.ml);
    p.logits = mass ? reinterpret_cast<float *>(sc + ds.logits) : nullptr;
    p.mass = mass; p.mass_out = mass_out; p.mass_cap = mass_cap;
    p.grid = ds.grid;
    p.by_row = ds.by_row;
    // At 0, 2, 3, 5 and 7 tiles: 24 sequences of 1 .. 8192 with 8 key heads 46.7, 26.0, 25.6, 26.0 and
    // 27.0 us (d = 128; 31.5, 18.4, 18.7, 19.4 and 20.2 at d = 64), 64 of 1 .. 20000 with 2 and weights 78.8,
    // 51.0, 49.2, 48.7 and 48.4 (53.4, 34.8, 34.1, 33.8 and 34.6), 7 of 301 .. 2500 with 16 and weights 20.0,
    // 17.6, 17.8, 18.6 and 19.9 (15.8, 14.4, 14.3, 15.2 and 15.9).
    p.row_cost = 3;
    p.word = static_cast<uint32_t *>(workspace);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == kDtypeBf16)
        return d == 64 ? launch_decode<__nv_bfloat16, 64>(p, s) : launch_decode<__nv_bfloat16, 128>(p, s);
    return d == 64 ? launch_decode<__half, 64>(p, s) : launch_decode<__half, 128>(p, s);
}

size_t streamkl_evict_scratch_size(int B, int H_k, int num_pages, int page_size, int max_pages, int mass_cap,
                                   int budget) {
    if (B <= 0 || H_k < 1 || num_pages < 0 || page_size < 1 || max_pages < 0 || mass_cap < 0 || budget < 0) return 0;
    return evict_scratch(B, H_k, num_pages, page_size, max_pages, mass_cap, budget).total;
}

streamkl_status streamkl_evict(void *k_pages, const long long *k_stride, void *v_pages, const long long *v_stride,
                               int B, int H_k, int d, int num_pages, int page_size, const int *page_table,
                               int max_pages, long long table_stride, const int *seq_len, const float *mass,
                               const int *pos, const int *next_pos, int mass_cap, int budget, int recent, int *new_len,
                               float *mass_out, int *pos_out, void *workspace, size_t workspace_bytes, void *scratch,
                               size_t scratch_bytes, void *stream) {
    if (!paged_shape_ok(B, H_k, H_k, num_pages, page_size, max_pages, kDtypeBf16)) return STREAMKL_ERR_INVALID_ARG;
    if (mass_cap < 0 || mass_cap > kMaxCap || budget < 0 || recent < 0 || recent > budget) return STREAMKL_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kWorkspaceBytes) return STREAMKL_ERR_WORKSPACE;
    if (!aligned16(workspace) || !aligned16(scratch)) return STREAMKL_ERR_INVALID_ARG;
    if (recent > 0 && (!pos || !next_pos)) return STREAMKL_ERR_INVALID_ARG;
    if ((pos == nullptr) != (pos_out == nullptr)) return STREAMKL_ERR_INVALID_ARG;
    if (B == 0) return STREAMKL_OK;
    const bool slots = mass_cap > 0;
    if (!aligned4(mass) || !aligned4(mass_out) || !aligned4(pos) || !aligned4(pos_out) || !aligned4(next_pos) ||
        !aligned4(new_len))
        return STREAMKL_ERR_INVALID_ARG;
    if (!seq_len || !new_len || new_len == seq_len) return STREAMKL_ERR_INVALID_ARG;
    if (num_pages > 0 && k_pages && k_pages == v_pages) return STREAMKL_ERR_INVALID_ARG;
    if (slots && (!mass || !mass_out || mass == mass_out || (pos && pos == pos_out))) return STREAMKL_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_pages, v_pages, num_pages, page_table, max_pages, seq_len)) return STREAMKL_ERR_INVALID_ARG;
    if ((long long)B * max_pages > 0x7fffffffll || (long long)num_pages * page_size > 0xffffffffll)
        return STREAMKL_ERR_INVALID_ARG;
    if (paged_cap(page_size, max_pages, seq_len, mass_cap) > kEvictMaxCluster * kEvictMaxWords * 32)
        return STREAMKL_ERR_UNSUPPORTED;
    const EvictScratch es = evict_scratch(B, H_k, num_pages, page_size, max_pages, mass_cap, budget);
    if (!scratch || scratch_bytes < es.total) return STREAMKL_ERR_WORKSPACE;
    const long long cont[3] = {(long long)H_k * page_size * d, (long long)page_size * d, d};
    const long long *ks = k_stride ? k_stride : cont, *vs = v_stride ? v_stride : cont;
    const long long pe[3] = {num_pages, H_k, page_size};
    if (!stride_ok(ks, pe) || !stride_ok(vs, pe)) return STREAMKL_ERR_INVALID_ARG;
    if (B > 1 && table_stride < 0) return STREAMKL_ERR_INVALID_ARG;
    // (keys and values may lie between each other: pages that hold both)
    const long long weights = (long long)B * H_k * mass_cap;
    const long long used[3] = {num_pages, H_k, std::min(page_size, paged_cap(page_size, max_pages, seq_len, mass_cap))};
    const Span keys = rows_span(k_pages, ks, used, d), values = rows_span(v_pages, vs, used, d);
    const Span table = table_span(page_table, B, max_pages, table_stride), lens = vec_span(seq_len, B);
    const Span m = vec_span(mass, weights), at = vec_span(pos, weights), next = vec_span(next_pos, B);
    if (overlapping({vec_span(new_len, B), vec_span(mass_out, weights), vec_span(pos_out, weights)},
                    {keys, values, table, lens, m, at, next}) ||
        overlapping({keys}, {table, lens, m, at, next}) || overlapping({values}, {table, lens, m, at, next}))
        return STREAMKL_ERR_INVALID_ARG;
    streamkl_status st = check_device();
    if (st != STREAMKL_OK) return st;

    EvictParams p;
    memset(&p, 0, sizeof p);
    p.B = B; p.Hk = H_k; p.d = d;
    p.pages = num_pages; p.page = page_size; p.max_pages = max_pages;
    p.cap = paged_cap(page_size, max_pages, scratch, mass_cap);
    p.k = PageView{k_pages, ks[0], ks[1], ks[2]};
    p.v = PageView{v_pages, vs[0], vs[1], vs[2]};
    p.table = page_table; p.table_b = table_stride; p.len = seq_len;
    p.mass = mass; p.pos = pos; p.next_pos = next_pos;
    p.mass_cap = mass_cap; p.budget = budget; p.recent = recent;
    p.new_len = new_len; p.mass_out = mass_out; p.pos_out = pos_out;
    char *sc = static_cast<char *>(scratch);
    p.owner = reinterpret_cast<int *>(sc + es.owner);
    p.refused = reinterpret_cast<int *>(sc + es.refused);
    p.moves = reinterpret_cast<int *>(sc + es.moves);
    p.lists = reinterpret_cast<int *>(sc + es.lists);
    p.list = es.list;
    p.word = static_cast<uint32_t *>(workspace);
    cudaStream_t s = (cudaStream_t)stream;
    // CTAs of a cluster: twice as many as long as each keeps over 8192 slots and there are no more
    // than SMs, so that up to two an SM are launched (both fit while each keeps up to 25 thousand slots);
    // four prompts of 32 thousand slots and 8 key heads: 60, 49 and 50 us with 2, 4 and 8
    const long long rows = (long long)B * H_k;
    int cs = 1;
    while (cs < kEvictMaxCluster && p.cap / cs > 8192 &&
           (rows * cs <= sm_count() || p.cap / cs > kEvictMaxWords * 32))
        cs *= 2;
    p.words = ((p.cap + 31) / 32 + cs - 1) / cs;
    if (set_smem(streamkl_evict_select_kernel, std::max(evict_smem(kEvictKeyWords), evict_smem(kEvictMaxWords))) !=
        cudaSuccess)
        return STREAMKL_ERR_CUDA;
    // a launch less where each sequence can look through the whole table itself
    p.claims = (long long)B * max_pages > kEvictTable;
    if (p.claims && (st = launch_ex(streamkl_evict_claim_kernel, B, 256, 0, s, false, 1, p)) != STREAMKL_OK) return st;
    st = launch_ex(streamkl_evict_select_kernel, rows * cs, kEvictThreads, evict_smem(p.words), s, p.claims != 0, cs, p, cs);
    if (st != STREAMKL_OK) return st;
    // blocks for one and a half times what runs at once (8 an SM): rows with nothing to move leave early
    const int per = 256 / (d / 4);
    const long long room = (12ll * std::max(1, sm_count()) + rows - 1) / rows;
    const int nx = (int)std::max(1ll, std::min<long long>(room, (p.list + per - 1) / per));
    return launch_ex(streamkl_evict_move_kernel, nx * rows, 256, 0, s, true, 1, p, nx);
}

}  // extern "C"
