// evict.cuh — eviction from a paged key-value cache by accumulated attention
// weight.  Of the n slots of (sequence, key head) the `keep` = min(n, budget)
// largest stay, ranked by
//     (recent, weight, lowest slot),   recent = pos >= next_pos - n_recent,
// and the kept tokens of the slots past `keep`, in order, fill the slots of
// the evicted ones before it.  Attention does not depend on the order of the
// slots, so this moves the fewest rows that leave the first `keep` slots full:
// one row when one token is evicted, where keeping the order would move half
// of the cache.  Sources lie past `keep` and targets before it, so no move
// reads what another writes.
//
// Weights are ranked as integers: the bits of a positive float grow with it,
// anything else (zero, negative, NaN) ranks as 0, recent ones above infinity.
// The keep-th largest is found by a radix selection, 8 bits at a time; ties at
// that value go to the lowest slots.
//
// Kernels, each started while the one before it runs:
//   claim   (tables of many entries) every used entry writes its number to its
//           page's owner word
//   select  a cluster of CTAs a (sequence, key head): selection, lists of moves,
//           compacted weights and positions; then the search for pages with a
//           second user: an entry that finds another's number in its page's owner
//           word, or (small tables) a sequence that finds a page of its own in
//           another's row of the table
//   move    the rows
// The bytes are few (8 a slot, 8 d a moved row), so what counts is the length
// of the chain of dependent steps: the slots of a long sequence are spread over
// up to 8 CTAs that add their histograms through distributed shared memory, and
// what is kept is a bit a slot, so that ranks come from one prefix sum over the
// words of 32 slots.  Measured: 11 us for one sequence of 1040, 20 us for 32 of
// 4160 (8 key heads), 51 us for 4 of 32768 to 4096 (selection 22, moves 27).
#pragma once

#include "decode.cuh"

namespace skl {

struct EvictParams {
    int B, Hk, d;
    int pages, page, max_pages, cap;     // cap: slots a sequence may have, min(max_pages * page, mass_cap)
    PageView k, v;
    const int *table, *len;
    long long table_b;
    const float *mass;                   // [B, Hk, mass_cap]
    const int *pos, *next_pos;           // [B, Hk, mass_cap], [B]; or null
    int mass_cap, budget, recent;
    int *new_len;                        // [B]
    float *mass_out;                     // [B, Hk, mass_cap]
    int *pos_out;                        // or null
    int claims;                          // pages are claimed by a kernel of their own
    int *owner;                          // [pages]: the last claimant's sequence * max_pages + table column
    int *refused;                        // [B]: 1 = the sequence is left as it is
    int *moves;                          // [B * Hk] number of moved rows
    int *lists;                          // [B * Hk][4][list] targets and sources: as rows of the cache
                                         // (page number * slots of a page + slot), and as slots
    int list;
    int words;                           // 32-slot words a CTA of the cluster keeps in shared memory
    uint32_t *word;
};

constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictKeyWords = 1024;                       // 32768 slots a CTA keeps the keys of (else it rereads)
constexpr int kEvictMaxWords = 8192;                       // and 262144 that it can deal with
constexpr int kEvictBins = 256, kEvictPasses = 4;          // a radix digit a pass
constexpr int kEvictMaxCluster = 8;

// Dynamic shared memory: a histogram a pass, three values a word of 32 slots, the keys.
__host__ __device__ constexpr int evict_smem(int words) {
    return kEvictPasses * kEvictBins * 4 + words * 3 * 4 + (words <= kEvictKeyWords ? words * 32 * 4 : 0);
}

__device__ __forceinline__ uint32_t weight_key(float m, bool recent) {
    return recent ? 0xffffffffu : (m > 0.f ? __float_as_uint(m) : 0u);
}

// Columns of the table that a sequence of n slots uses.  (A page may be as large as
// 2^31 - 1 slots, so n + page - 1 would overflow, and no page would be looked at.)
__host__ __device__ constexpr int used_pages(int n, int page) { return n > 0 ? (n - 1) / page + 1 : 0; }
static_assert(used_pages(0, 1) == 0 && used_pages(1, 16) == 1 && used_pages(16, 16) == 1 && used_pages(17, 16) == 2 &&
                  used_pages(2, 0x7fffffff) == 1 && used_pages(1 << 21, 0x7fffffff) == 1 &&
                  used_pages(1 << 21, 1) == 1 << 21,
              "no sum leaves 32 bits");

__global__ void __launch_bounds__(256) streamkl_evict_claim_kernel(const EvictParams p) {
    grid_release();
    const int b = blockIdx.x;
    if (threadIdx.x == 0) p.refused[b] = 0;
    const int n = cache_len(p.len, b, p.cap, p.word, threadIdx.x == 0), np = used_pages(n, p.page);
    for (int x = threadIdx.x; x < np; x += 256) {
        if (!bound_ok(x < p.max_pages, p.word, kSiteTable)) break;
        const int pg = __ldg(p.table + (size_t)b * p.table_b + x);
        if ((unsigned)pg < (unsigned)p.pages) p.owner[pg] = b * p.max_pages + x;
    }
}

// Exclusive prefix sums over the block of two counters a thread, and their
// totals.  `sh`: two words a warp, not in use by a scan that some thread may
// still read.
__device__ __forceinline__ int2 evict_scan(int2 x, int2 *sh, int2 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v.x, o), z = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) { v.x += y; v.y += z; }
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    const int2 t = lane < kEvictWarps ? sh[lane] : make_int2(0, 0);
    total = make_int2(__reduce_add_sync(0xffffffffu, t.x), __reduce_add_sync(0xffffffffu, t.y));
    return make_int2(v.x - x.x + __reduce_add_sync(0xffffffffu, lane < warp ? t.x : 0),
                     v.y - x.y + __reduce_add_sync(0xffffffffu, lane < warp ? t.y : 0));
}

// A cluster of `cs` CTAs a (sequence, key head).
__global__ void __launch_bounds__(kEvictThreads, 2) streamkl_evict_select_kernel(const EvictParams p, int cs) {
    extern __shared__ __align__(16) int evict_sh[];
    int *hist = evict_sh;                                  // [kEvictPasses][kEvictBins]
    uint32_t *kept_sh = reinterpret_cast<uint32_t *>(evict_sh + kEvictPasses * kEvictBins);
    uint32_t *hole_sh = kept_sh + p.words, *mover_sh = hole_sh + p.words, *keys_sh = mover_sh + p.words;
    __shared__ int2 scan_sh[2][kEvictWarps];
    __shared__ int cta_sh[3];                              // ties, holes, movers of the CTA, read by the cluster
    __shared__ uint32_t prefix_sh;
    __shared__ int want_sh, done_sh, refuse_sh;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    const int bk = blockIdx.x / cs, b = bk / p.Hk, hk = bk % p.Hk, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    grid_release();
    const int n = cache_len(p.len, b, p.cap, p.word, !p.claims && hk == 0 && tid == 0), keep = min(n, p.budget);
    const float *mass = p.mass + (size_t)bk * p.mass_cap;
    const int *pos = p.pos ? p.pos + (size_t)bk * p.mass_cap : nullptr;
    float *mass_out = p.mass_out + (size_t)bk * p.mass_cap;
    int *pos_out = p.pos_out ? p.pos_out + (size_t)bk * p.mass_cap : nullptr;
    int *to = p.lists + (size_t)bk * 4 * p.list, *from = to + p.list;
    int *to_slot = from + p.list, *from_slot = to_slot + p.list;

    // slots that no token is left in
    for (int t = n + rank * kEvictThreads + tid; t < p.mass_cap; t += cs * kEvictThreads) {
        mass_out[t] = 0.f;
        if (pos_out) pos_out[t] = -1;
    }
    const long long cut = p.recent > 0 ? (long long)__ldg(p.next_pos + b) - p.recent : 0;
    // this CTA's words of 32 slots
    const int words = (n + 31) / 32, per = (words + cs - 1) / cs;
    const int w0 = min(words, rank * per), nw = min(words, w0 + per) - w0;
    const int slots = min(n, (w0 + nw) * 32) - w0 * 32;    // and its slots, from 32 w0
    const bool in_smem = p.words <= kEvictKeyWords;
    if (tid < kEvictPasses * kEvictBins / 4) reinterpret_cast<int4 *>(hist)[tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
    // One pass over the slots: the keys, the first histogram, and every value
    // to its own slot (targets of moves are overwritten at the end).
    constexpr int U = 4;
    for (int x0 = tid; x0 < slots; x0 += U * kEvictThreads) {
        float m[U];
        int q[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int x = x0 + k * kEvictThreads, t = w0 * 32 + x;
            m[k] = x < slots ? mass[t] : 0.f;
            q[k] = x < slots && pos ? pos[t] : 0;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int x = x0 + k * kEvictThreads, t = w0 * 32 + x;
            if (x >= slots) break;
            if (!bound_ok(t < p.mass_cap, p.word, kSiteSlot)) break;
            mass_out[t] = t < keep ? m[k] : 0.f;
            if (pos_out) pos_out[t] = t < keep ? q[k] : -1;
            if (keep == n) continue;
            const uint32_t key = weight_key(m[k], p.recent > 0 && q[k] >= cut);
            if (in_smem) keys_sh[x] = key;
            atomicAdd(&hist[key >> 24], 1);
        }
    }
    if (n == keep) {                                       // nothing to evict (the whole cluster)
        if (tid == 0 && rank == 0) p.moves[bk] = 0;
    } else {
        auto key_of = [&](int x) -> uint32_t {
            const int t = w0 * 32 + x;
            return in_smem ? keys_sh[x] : weight_key(mass[t], p.recent > 0 && pos[t] >= cut);
        };
        // the keep-th largest key, a digit a pass (keep = 0: none is kept),
        // until the keys that share its digits are all wanted
        uint32_t prefix = 0xffffffffu;
        int want = keep;
        bool done = false;
#pragma unroll
        for (int pass = 0; pass < kEvictPasses && !done; ++pass) {
            const int shift = 24 - 8 * pass;
            int *h = hist + pass * kEvictBins;
            if (pass > 0)
                for (int x = tid; x < slots; x += kEvictThreads) {
                    const uint32_t key = key_of(x);
                    if (((key ^ prefix) >> (shift + 8)) == 0) atomicAdd(&h[(key >> shift) & 255u], 1);
                }
            if (cs > 1) cluster_sync(); else __syncthreads();
            // digits from the largest down, eight a lane of one warp
            int c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = 0;
            const int *mine = h + kEvictBins - 8 - 8 * lane;
            if (warp == 0) {
                if (cs > 1) {
#pragma unroll
                    for (int r0 = 0; r0 < kEvictMaxCluster; r0 += 4) {
                        if (r0 >= cs) break;
                        int4 y[8];                         // four ranks' loads in flight
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t at = cluster_addr(mine, min(r0 + r, cs - 1));
                            y[2 * r] = ld_cluster_v4(at);
                            y[2 * r + 1] = ld_cluster_v4(at + 16);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (r0 + r >= cs) break;
                            c[0] += y[2 * r].x; c[1] += y[2 * r].y; c[2] += y[2 * r].z; c[3] += y[2 * r].w;
                            c[4] += y[2 * r + 1].x; c[5] += y[2 * r + 1].y; c[6] += y[2 * r + 1].z;
                            c[7] += y[2 * r + 1].w;
                        }
                    }
                } else {
                    const int4 y0 = *reinterpret_cast<const int4 *>(mine), y1 = *reinterpret_cast<const int4 *>(mine + 4);
                    c[0] = y0.x; c[1] = y0.y; c[2] = y0.z; c[3] = y0.w;
                    c[4] = y1.x; c[5] = y1.y; c[6] = y1.z; c[7] = y1.w;
                }
                int sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += c[e];
                int v = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += y;
                }
                int before = v - sum;
#pragma unroll
                for (int e = 7; e >= 0; --e) {             // bin 255 - 8 lane - 7 + e
                    if (want > before && want <= before + c[e]) {
                        prefix_sh = (uint32_t)(kEvictBins - 8 - 8 * lane + e) << shift;
                        want_sh = want - before;
                        done_sh = want - before == c[e];
                    }
                    before += c[e];
                }
            }
            __syncthreads();
            if (keep > 0) {
                prefix = (pass == 0 ? 0u : prefix) | prefix_sh;
                want = want_sh;
                done = done_sh && prefix > 0u;
            }
        }
        if (done) {                                        // every key from `prefix` on, and no ties
            prefix -= 1u;
            want = 0;
        }
        // Kept: keys above `prefix`, and the first `want` slots that equal it.
        // Masks of a word of slots by a warp (ties for now in hole_sh) ...
        for (int w = warp; w < nw; w += kEvictWarps) {
            const int x = w * 32 + lane;
            const uint32_t key = x < slots ? key_of(x) : 0u;
            const uint32_t above = __ballot_sync(0xffffffffu, keep > 0 && x < slots && key > prefix);
            const uint32_t tie = __ballot_sync(0xffffffffu, keep > 0 && x < slots && key == prefix);
            if (lane == 0) {
                kept_sh[w] = above;
                hole_sh[w] = tie;
            }
        }
        __syncthreads();
        // ... then counts by a thread a run of words
        const int wt = (nw + kEvictThreads - 1) / kEvictThreads, v0 = min(nw, tid * wt), v1 = min(nw, v0 + wt);
        // sum of counter c over the lower ranks, and over all (a lane a rank)
        auto of_ranks = [&](int c, int &all) -> int {
            const int v = lane < cs ? (cs > 1 ? ld_cluster(cluster_addr(&cta_sh[c], lane)) : cta_sh[c]) : 0;
            all = __reduce_add_sync(0xffffffffu, v);
            return __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
        };
        int2 count = make_int2(0, 0), total;
        for (int w = v0; w < v1; ++w) count.x += __popc(hole_sh[w]);
        int tie_at = evict_scan(count, scan_sh[0], total).x, all;
        if (cs > 1) {
            if (tid == 0) cta_sh[0] = total.x;
            cluster_sync();
            tie_at += of_ranks(0, all);
        }
        count = make_int2(0, 0);
        for (int w = v0; w < v1; ++w) {
            const uint32_t tie = hole_sh[w];
            const int ties = __popc(tie), room = min(max(want - tie_at, 0), ties);
            uint32_t out = tie;                            // the word's ties past the room
            if (room == ties) out = 0u;
            else for (int k = 0; k < room; ++k) out &= out - 1u;
            tie_at += ties;
            const uint32_t kept = kept_sh[w] | (tie & ~out);
            const int left = keep - (w0 + w) * 32;         // slots of the word below the new length
            const uint32_t low = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
            kept_sh[w] = kept;
            count.x += __popc(low & ~kept);
            count.y += __popc(kept & ~low);
        }
        int2 at = evict_scan(count, scan_sh[1], total);
        if (tid == 0) {
            cta_sh[1] = total.x;
            cta_sh[2] = total.y;
        }
        if (cs > 1) cluster_sync(); else __syncthreads();
        int n_moves;                                       // of the whole cluster
        at.y += of_ranks(2, all);
        at.x += of_ranks(1, n_moves);
        for (int w = v0; w < v1; ++w) {
            const int left = keep - (w0 + w) * 32;
            const uint32_t low = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u), kept = kept_sh[w];
            hole_sh[w] = (uint32_t)at.x;
            mover_sh[w] = (uint32_t)at.y;
            at.x += __popc(low & ~kept);
            at.y += __popc(kept & ~low);
        }
        __syncthreads();
        for (int w = warp; w < nw; w += kEvictWarps) {
            const int t = (w0 + w) * 32 + lane;
            const uint32_t kept = kept_sh[w], low = __ballot_sync(0xffffffffu, t < keep), below = (1u << lane) - 1u;
            const uint32_t hole = low & ~kept, mover = kept & ~low;
            const bool is_hole = (hole >> lane) & 1, is_mover = (mover >> lane) & 1;
            if (!is_hole && !is_mover) continue;
            // the cache's row (a bad page's is never used: the sequence is refused)
            const unsigned at_page = (unsigned)t / (unsigned)p.page;
            if (!bound_ok(at_page < (unsigned)p.max_pages && t < p.mass_cap, p.word, kSiteTable)) continue;
            const int row = (int)((unsigned)__ldg(p.table + (size_t)b * p.table_b + at_page) * (unsigned)p.page +
                                  ((unsigned)t - at_page * (unsigned)p.page));
            if (is_hole) {
                const int x = (int)hole_sh[w] + __popc(hole & below);
                if (!bound_ok(x >= 0 && x < p.list, p.word, kSiteList)) continue;
                to[x] = row;
                to_slot[x] = t;
            } else {
                const int x = (int)mover_sh[w] + __popc(mover & below);
                if (!bound_ok(x >= 0 && x < p.list, p.word, kSiteList)) continue;
                from[x] = row;
                from_slot[x] = t;
            }
        }
        if (tid == 0 && rank == 0) p.moves[bk] = n_moves;
        if (cs > 1) cluster_sync(); else __syncthreads();  // the lists are whole
        for (int x = rank * kEvictThreads + tid; x < n_moves; x += cs * kEvictThreads) {
            if (!bound_ok(x < p.list, p.word, kSiteList)) break;
            const int t = to_slot[x], f = from_slot[x];
            if (!bound_ok(t >= 0 && t < keep && f >= keep && f < n, p.word, kSiteSlot)) continue;
            mass_out[t] = mass[f];
            if (pos_out) pos_out[t] = pos[f];
        }
    }
    grid_wait();                                           // every claim is made
    if (hk != 0) return;
    if (tid == 0 && rank == 0) p.new_len[b] = keep;
    if (!p.claims) {
        // A sequence with a page out of range, or that evicts or meets one that
        // does over a common page, refuses itself (and the other does the same).
        // A bit a page (modulo 32768) sorts out nearly all of the others' entries.
        if (rank != 0) return;
        const int np = used_pages(n, p.page);
        const int *row = p.table + (size_t)b * p.table_b;
        auto own = [&](int pg, int but) -> bool {
            for (int y = 0; y < np; ++y)
                if (y != but && __ldg(row + y) == pg) return true;
            return false;
        };
        __syncthreads();
        for (int x = tid; x < kEvictPasses * kEvictBins; x += kEvictThreads) hist[x] = 0;
        if (tid == 0) refuse_sh = 0;
        __syncthreads();
        static_assert(kEvictPasses * kEvictBins * 32 == 32768, "bits of the histograms' memory");
        uint32_t why = 0u;
        for (int x = tid; x < np; x += kEvictThreads) {
            if (!bound_ok(x < p.max_pages, p.word, kSiteTable)) break;
            const int pg = __ldg(row + x);
            if ((unsigned)pg >= (unsigned)p.pages) {
                why |= kStatusBadPage;
                continue;
            }
            const int was = atomicOr(&hist[(pg & 32767) >> 5], 1 << (pg & 31));
            if (n > keep && ((was >> (pg & 31)) & 1) && own(pg, x)) why |= kStatusSharedPage;
        }
        __syncthreads();
        for (int e = tid; e < p.B * p.max_pages; e += kEvictThreads) {
            const int ob = e / p.max_pages, x = e - ob * p.max_pages;
            if (ob == b) continue;
            const int on = cache_len(p.len, ob, p.cap, p.word, false);
            if ((long long)x * p.page >= on || (n <= keep && on <= p.budget)) continue;
            const int pg = __ldg(p.table + (size_t)ob * p.table_b + x);
            if ((unsigned)pg < (unsigned)p.pages && ((hist[(pg & 32767) >> 5] >> (pg & 31)) & 1) && own(pg, -1))
                why |= kStatusSharedPage;
        }
        if (why) {
            if (p.word) atomicOr(p.word, why);
            refuse_sh = 1;
        }
        __syncthreads();
        if (tid == 0) p.refused[b] = refuse_sh;
        return;
    }
    // Of the users of a page all but the last claimant find its number: each
    // that evicts, or meets one that does, is refused, and so is that one.
    const int np = used_pages(n, p.page);
    for (int x = rank * kEvictThreads + tid; x < np; x += cs * kEvictThreads) {
        if (!bound_ok(x < p.max_pages, p.word, kSiteTable)) break;
        const int pg = __ldg(p.table + (size_t)b * p.table_b + x);
        if ((unsigned)pg >= (unsigned)p.pages) {
            if (p.word) atomicOr(p.word, (uint32_t)kStatusBadPage);
            p.refused[b] = 1;
            continue;
        }
        const int other = p.owner[pg];
        if (other == b * p.max_pages + x) continue;
        const int ob = other / p.max_pages, on = cache_len(p.len, ob, p.cap, p.word, false);
        if (n > keep || on > min(on, p.budget)) {
            if (p.word) atomicOr(p.word, (uint32_t)kStatusSharedPage);
            p.refused[b] = 1;
            p.refused[ob] = 1;
        }
    }
}

// Moves the rows; nx blocks a (sequence, key head).  A sequence whose pages
// were found shared or out of range is put back to what it was: length,
// weights and positions copied, no row moved.
// (More CTAs, not more rows in flight a thread: 63 us with four, 51 with one.)
__global__ void __launch_bounds__(256, 8) streamkl_evict_move_kernel(const EvictParams p, int nx) {
    const int bk = blockIdx.x / nx, bx = blockIdx.x % nx, b = bk / p.Hk, hk = bk % p.Hk;
    grid_wait();
    if (p.refused[b]) {
        const int n = cache_len(p.len, b, p.cap, p.word, false);
        if (hk == 0 && bx == 0 && threadIdx.x == 0) p.new_len[b] = n;
        for (int t = bx * 256 + threadIdx.x; t < p.mass_cap; t += nx * 256) {
            const size_t at = (size_t)bk * p.mass_cap + t;
            p.mass_out[at] = t < n ? p.mass[at] : 0.f;
            if (p.pos_out) p.pos_out[at] = t < n ? p.pos[at] : -1;
        }
        return;
    }
    const int m = p.moves[bk];
    const int ch = p.d / 8;                                // 16-byte chunks in a row; 2 ch lanes move a K and a V row
    const int per = 256 / (2 * ch);                        // tokens a block moves at a time
    const int *to = p.lists + (size_t)bk * 4 * p.list, *from = to + p.list;
    const int x = threadIdx.x % (2 * ch);
    const PageView pv = x < ch ? p.k : p.v;
    uint16_t *base = static_cast<uint16_t *>(const_cast<void *>(pv.ptr)) + hk * pv.s_head + (x % ch) * 8;
    auto row = [&](unsigned r) -> uint16_t * {
        const unsigned pg = r / (unsigned)p.page;
        return base + (long long)pg * pv.s_page + (long long)(r - pg * (unsigned)p.page) * pv.s_slot;
    };
    const int step = nx * per;
    int r = bx * per + (int)(threadIdx.x / (2 * ch));
    unsigned t = r < m ? to[r] : 0u, f = r < m ? from[r] : 0u;
    while (r < m) {
        const unsigned td = t, fd = f;
        r += step;
        if (r < m) { t = to[r]; f = from[r]; }             // the next pair while this row travels
        if (!bound_ok(r - step < p.list && td / (unsigned)p.page < (unsigned)p.pages &&
                          fd / (unsigned)p.page < (unsigned)p.pages,
                      p.word, kSiteSlot))
            continue;
        *reinterpret_cast<uint4 *>(row(td)) = *reinterpret_cast<const uint4 *>(row(fd));
    }
}

}  // namespace skl
