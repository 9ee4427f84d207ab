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

// 4-D map over rows of d elements in [n3][n2][n1][d] with strides (in
// elements) s3, s2, s1: box of 64 columns x `rows` rows, 128-byte swizzle,
// zeros outside, so ragged tiles read zeros.
bool make_rows_map(CUtensorMap *m, const void *ptr, int d, int n1, int n2, int n3, long long s1, long long s2,
                   long long s3, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t any = (cuuint64_t)d * 2;        // stride of a dimension with one element
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
    cuuint64_t strides[3] = {n1 > 1 ? (cuuint64_t)s1 * 2 : any, n2 > 1 ? (cuuint64_t)s2 * 2 : any,
                             n3 > 1 ? (cuuint64_t)s3 * 2 : any};
    cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pieces that a streamed range of at most `tiles` tiles is cut into when there
// are `items` owned tiles for two CTAs an SM: as key_splits above.
int stat_splits(long long items, long long tiles) {
    const long long slots = 2ll * sm_count();
    if (slots <= 0 || items == 0 || items >= 4 * slots) return 1;
    const int smax = (int)std::min<long long>(kMaxSplits, tiles / kMinSplitTiles);
    int best = 1;
    double best_t = 1e300;
    for (int S = 1; S <= std::max(1, smax); ++S) {
        const double t = (double)((items * S + slots - 1) / slots) / S * (1.0 + 0.02 * (S - 1));
        if (t < best_t * (1.0 - 1e-9)) { best = S; best_t = t; }
    }
    return best;
}

struct StatPlan {
    long long lse_items, mass_items;
    int lse_splits, mass_splits;
    size_t bytes;                    // scratch of the splits
};

StatPlan stat_plan(int B, int H, int Hk, int N_Q, int N_K, bool lse_given) {
    StatPlan s;
    const long long G = H / Hk;
    s.lse_items = (long long)B * Hk * ((G * N_Q + 127) / 128);
    s.mass_items = (long long)B * Hk * ((N_K + 127) / 128);
    s.lse_splits = lse_given ? 1 : stat_splits(s.lse_items, (N_K + 63) / 64);
    s.mass_splits = stat_splits(s.mass_items, G * ((N_Q + 63) / 64));
    const size_t a = s.lse_splits > 1 ? (size_t)s.lse_splits * 2 * B * H * N_Q * sizeof(float) : 0;
    const size_t b = s.mass_splits > 1 ? (size_t)s.mass_splits * B * Hk * N_K * sizeof(float) : 0;
    s.bytes = std::max(a, b);
    return s;
}

bool stat_shape_ok(int B, int H, int H_k, int N_Q, int N_K, int d, int dtype, int causal) {
    if (B < 0 || H < 0 || N_Q < 0 || N_K < 0 || H_k < 1 || (H > 0 && H % H_k != 0)) return false;
    if (causal != 0 && causal != 1) return false;
    if (causal && N_Q > N_K) return false;
    if (!causal && N_K == 0 && N_Q > 0 && B > 0 && H > 0) return false;
    if (dtype != kDtypeBf16 && dtype != kDtypeFp16) return false;
    return (long long)B * H <= (1ll << 24) && (long long)B * H_k <= (1ll << 24) && N_Q <= (1 << 24) && N_K <= (1 << 24) &&
           (long long)H * N_Q < (1ll << 31);
}

template <int D, int MODE>
streamkl_status launch_stat(const CUtensorMap &map, StatParams p, long long items, float *part, size_t part_bytes,
                            int splits, cudaStream_t s) {
    const long long rows = MODE == kRowLse ? (long long)p.B * p.H * p.N_Q : (long long)p.B * p.Hk * p.N_K;
    const size_t need = (size_t)splits * (MODE == kRowLse ? 2 : 1) * rows * sizeof(float);
    p.splits = splits > 1 && part && part_bytes >= need ? splits : 1;
    p.part = part;
    if (items * p.splits > 0x7fffffffll) return STREAMKL_ERR_INVALID_ARG;
    auto kern = streamkl_stat_kernel<D, MODE>;
    if (set_smem(kern, StatCfg<D>::SMEM) != cudaSuccess) return STREAMKL_ERR_CUDA;
    kern<<<(unsigned)(items * p.splits), StatCfg<D>::THREADS, StatCfg<D>::SMEM, s>>>(map, p);
    if (cudaGetLastError() != cudaSuccess) return STREAMKL_ERR_CUDA;
    if (p.splits > 1) {
        const unsigned blocks = (unsigned)((rows + 255) / 256);
        if (MODE == kRowLse)
            streamkl_lse_merge_kernel<<<blocks, 256, 0, s>>>(p.part, p.splits, rows, p.lse);
        else
            streamkl_mass_sum_kernel<<<blocks, 256, 0, s>>>(p.part, p.splits, rows, p.accumulate, p.mass);
        if (cudaGetLastError() != cudaSuccess) return STREAMKL_ERR_CUDA;
    }
    return STREAMKL_OK;
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

int paged_cap(int page_size, int max_pages, const void *mass, int mass_cap) {
    long long cap = std::min<long long>((long long)page_size * max_pages, kMaxCap);
    if (mass) cap = std::min<long long>(cap, mass_cap);
    return (int)cap;
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
    return cudaLaunchKernelEx(&c, kern, args...) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
}

struct DecodeScratch {
    int grid;
    bool by_row;
    size_t o, ml, logits, total;     // byte offsets and the whole
};

// Sequences of at most this many slots are not split: a CTA streams a whole
// row, and there is no second kernel.
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
    const bool mass = p.logits && !(p.by_row && p.nhb == 1);
    if (st != STREAMKL_OK || (p.by_row && !mass)) return st;
    const long long n_join = p.by_row ? 0 : ((long long)p.B * p.H + 3) / 4;
    const int nx = std::max(1, (p.mass_cap + kFinishTokens - 1) / kFinishTokens);
    const long long n_mass = mass ? (long long)nx * p.B * p.Hk : 0;
    return launch_ex(streamkl_decode_finish_kernel<T, D>, n_join + n_mass, 128, 0, s, true, 1, p, (int)n_join, nx);
}

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
    if (B <= 0 || H <= 0 || H_k < 1 || H % H_k != 0 || N_Q <= 0 || N_K <= 0) return 0;
    return stat_plan(B, H, H_k, N_Q, N_K, lse_given != 0).bytes;
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
    streamkl_status st = check_device();
    if (st != STREAMKL_OK) return st;

    CUtensorMap mq, mk;
    if (!make_rows_map(&mq, q, d, N_Q, H, B, qs[2], qs[1], qs[0], 64) ||
        !make_rows_map(&mk, k, d, N_K, H_k, B, ks[2], ks[1], ks[0], 64))
        return STREAMKL_ERR_CUDA;
    const StatPlan plan = stat_plan(B, H, H_k, N_Q, N_K, lse_given != 0);
    StatParams p;
    memset(&p, 0, sizeof p);
    p.B = B; p.H = H; p.Hk = H_k; p.G = H / H_k; p.N_Q = N_Q; p.N_K = N_K; p.causal = causal;
    p.kv_len = kv_len;
    p.c = scale * kLog2e;
    p.idesc = dtype == kDtypeBf16 ? idesc_bf16(128, 64, 0, 0) : idesc_fp16(128, 64, 0, 0);
    p.lse = lse; p.mass = mass; p.accumulate = accumulate;
    p.st.word = static_cast<uint32_t *>(workspace);
    p.st.budget_ns = kWaitBudgetNs;
    float *part = static_cast<float *>(scratch);
    if (!lse_given) {
        p.own = q; p.own_b = qs[0]; p.own_h = qs[1]; p.own_n = qs[2];
        p.n_own = (int)(((long long)p.G * N_Q + 127) / 128);
        st = d == 64 ? launch_stat<64, kRowLse>(mk, p, plan.lse_items, part, scratch_bytes, plan.lse_splits, s)
                     : launch_stat<128, kRowLse>(mk, p, plan.lse_items, part, scratch_bytes, plan.lse_splits, s);
        if (st != STREAMKL_OK) return st;
    }
    p.own = k; p.own_b = ks[0]; p.own_h = ks[1]; p.own_n = ks[2];
    p.n_own = (N_K + 127) / 128;
    return d == 64 ? launch_stat<64, kKeyMass>(mq, p, plan.mass_items, part, scratch_bytes, plan.mass_splits, s)
                   : launch_stat<128, kKeyMass>(mq, p, plan.mass_items, part, scratch_bytes, plan.mass_splits, s);
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
    if ((long long)B * H == 0) return STREAMKL_OK;
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
    p.row_cost = d == 64 ? 3 : 2;
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
    const EvictScratch es = evict_scratch(B, H_k, num_pages, page_size, max_pages, mass_cap, budget);
    if (!scratch || scratch_bytes < es.total) return STREAMKL_ERR_WORKSPACE;
    const long long cont[3] = {(long long)H_k * page_size * d, (long long)page_size * d, d};
    const long long *ks = k_stride ? k_stride : cont, *vs = v_stride ? v_stride : cont;
    const long long pe[3] = {num_pages, H_k, page_size};
    if (!stride_ok(ks, pe) || !stride_ok(vs, pe)) return STREAMKL_ERR_INVALID_ARG;
    if (B > 1 && table_stride < 0) return STREAMKL_ERR_INVALID_ARG;
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
    // CTAs of a cluster: twice as many as long as each keeps over 2048 slots and all run at once
    const long long rows = (long long)B * H_k;
    int cs = 1;
    while (cs < kEvictMaxCluster && p.cap / cs > 2048 &&
           (rows * cs <= sm_count() || p.cap / cs > kEvictMaxWords * 32))
        cs *= 2;
    p.words = ((p.cap + 31) / 32 + cs - 1) / cs;
    if (p.words > kEvictMaxWords) return STREAMKL_ERR_UNSUPPORTED;
    if (set_smem(streamkl_evict_select_kernel, std::max(evict_smem(kEvictKeyWords), evict_smem(kEvictMaxWords))) !=
        cudaSuccess)
        return STREAMKL_ERR_CUDA;
    st = launch_ex(streamkl_evict_claim_kernel, B, 256, 0, s, false, 1, p);
    if (st != STREAMKL_OK) return st;
    st = launch_ex(streamkl_evict_select_kernel, rows * cs, kEvictThreads, evict_smem(p.words), s, true, cs, p, cs);
    if (st != STREAMKL_OK) return st;
    // blocks for one and a half times what runs at once (8 an SM): rows with nothing to move leave early
    const int per = 256 / (d / 4);
    const long long room = (12ll * std::max(1, sm_count()) + rows - 1) / rows;
    const int nx = (int)std::max(1ll, std::min<long long>(room, (p.list + per - 1) / per));
    return launch_ex(streamkl_evict_move_kernel, nx * rows, 256, 0, s, true, 1, p, nx);
}

}  // extern "C"
