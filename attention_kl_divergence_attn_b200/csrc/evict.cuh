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
// The keep-th largest is found by a radix selection, 11, 11 and 10 bits at a
// time; ties at that value go to the lowest slots.
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
    int *owner;                          // [pages] cleared to -1: 2 * sequence that uses a page + 1 if it evicts
    int *refused;                        // [B] cleared to -1: 0 = the sequence is left as it is
    int *moves;                          // [B * Hk] number of moved rows
    int *lists;                          // [B * Hk][2][list] targets, then sources
    int list;
    uint32_t *word;
};

constexpr int kEvictThreads = 1024;
constexpr int kEvictSmemKeys = 48 * 1024;                  // keys held in shared memory (longer caches are reread)

__device__ __forceinline__ uint32_t weight_key(float m, bool recent) {
    return recent ? 0xffffffffu : (m > 0.f ? __float_as_uint(m) : 0u);
}

// Exclusive prefix sum over the block of two counters packed in 64 bits;
// `total` is the block's sum.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long *sh,
                                                         unsigned long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    if (warp == 0) {
        unsigned long long w = lane < (int)(blockDim.x >> 5) ? sh[lane] : 0ull;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        sh[lane] = w;
    }
    __syncthreads();
    total = sh[(blockDim.x >> 5) - 1];
    const unsigned long long before = (warp ? sh[warp - 1] : 0ull) + v - x;
    __syncthreads();
    return before;
}

// One CTA a (sequence, key head): finds the kept slots, writes the moves and
// the compacted weights and positions.  Key head 0's CTA also claims the
// sequence's pages, to find pages that two sequences (or one twice) use.
__global__ void __launch_bounds__(kEvictThreads, 1) streamkl_evict_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys_sh[];
    __shared__ int hist[2048];
    __shared__ unsigned long long scan_sh[32];
    __shared__ uint32_t prefix_sh;
    __shared__ int want_sh;
    const int bk = blockIdx.x, b = bk / p.Hk, hk = bk % p.Hk, tid = threadIdx.x;
    const int n = cache_len(p.len, b, p.cap, p.word, tid == 0 && hk == 0);
    const int keep = min(n, p.budget);
    const float *mass = p.mass + (size_t)bk * p.mass_cap;
    const int *pos = p.pos ? p.pos + (size_t)bk * p.mass_cap : nullptr;
    float *mass_out = p.mass_out + (size_t)bk * p.mass_cap;
    int *pos_out = p.pos_out ? p.pos_out + (size_t)bk * p.mass_cap : nullptr;
    const long long cut = p.recent > 0 ? (long long)__ldg(p.next_pos + b) - p.recent : 0;
    int *to = p.lists + (size_t)bk * 2 * p.list, *from = to + p.list;

    if (hk == 0) {
        if (tid == 0) p.new_len[b] = keep;
        const int np = (n + p.page - 1) / p.page;
        for (int x = tid; x < np; x += kEvictThreads) {
            const int pg = __ldg(p.table + (size_t)b * p.table_b + x);
            if ((unsigned)pg >= (unsigned)p.pages) {
                if (p.word) atomicOr(p.word, (uint32_t)kStatusBadPage);
                p.refused[b] = 0;
            } else {
                // every user of a page passes here in some order, so one that
                // evicts meets the one before or the one after it
                const int me = 2 * b + (n > keep ? 1 : 0), was = atomicExch(p.owner + pg, me);
                if (was >= 0 && ((was | me) & 1)) {
                    if (p.word) atomicOr(p.word, (uint32_t)kStatusSharedPage);
                    p.refused[b] = 0;
                    p.refused[was >> 1] = 0;
                }
            }
        }
    }
    if (n <= keep) {                                       // nothing to evict
        if (tid == 0) p.moves[bk] = 0;
        for (int t = tid; t < p.mass_cap; t += kEvictThreads) {
            mass_out[t] = t < n ? mass[t] : 0.f;
            if (pos_out) pos_out[t] = t < n ? pos[t] : -1;
        }
        return;
    }
    const bool in_smem = n <= kEvictSmemKeys;
    auto key_at = [&](int t) -> uint32_t {
        return weight_key(mass[t], p.recent > 0 && pos[t] >= cut);
    };
    if (in_smem)
        for (int t = tid; t < n; t += kEvictThreads) keys_sh[t] = key_at(t);
    // radix selection of the keep-th largest key
    uint32_t prefix = 0, mask = 0;
    int want = keep;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int x = tid; x < 2048; x += kEvictThreads) hist[x] = 0;
        __syncthreads();
        for (int t = tid; t < n; t += kEvictThreads) {
            const uint32_t key = in_smem ? keys_sh[t] : key_at(t);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1 << bits) - 1)], 1);
        }
        __syncthreads();
        // digits from the largest down: thread tid holds digits 2047 - 2 tid and the one below
        const int d1 = hist[2047 - 2 * tid], d0 = hist[2046 - 2 * tid];
        unsigned long long total;
        const int before = (int)block_scan((unsigned long long)(d1 + d0), scan_sh, total);
        if (want > before && want <= before + d1) {
            prefix_sh = prefix | ((uint32_t)(2047 - 2 * tid) << shift);
            want_sh = want - before;
        } else if (want > before + d1 && want <= before + d1 + d0) {
            prefix_sh = prefix | ((uint32_t)(2046 - 2 * tid) << shift);
            want_sh = want - before - d1;
        }
        __syncthreads();
        if (keep > 0) {
            prefix = prefix_sh;
            want = want_sh;
        }
        mask |= ((1u << bits) - 1u) << shift;
        __syncthreads();
    }
    // kept: keys above `prefix`, and the first `want` slots that equal it
    int ties = 0, holes = 0, movers = 0;
    for (int t0 = 0; t0 < n; t0 += kEvictThreads) {
        const int t = t0 + tid;
        const uint32_t key = t < n ? (in_smem ? keys_sh[t] : key_at(t)) : 0u;
        const bool tie = t < n && keep > 0 && key == prefix;
        unsigned long long total;
        const int tie_rank = ties + (int)block_scan(tie ? 1ull : 0ull, scan_sh, total);
        ties += (int)total;
        const bool kept = t < n && keep > 0 && (key > prefix || (tie && tie_rank < want));
        const bool hole = t < keep && !kept, mover = kept && t >= keep;
        const unsigned long long rank = block_scan((hole ? 1ull : 0ull) | (mover ? 1ull << 32 : 0ull), scan_sh, total);
        if (hole) to[holes + (int)(rank & 0xffffffffull)] = t;
        if (mover) from[movers + (int)(rank >> 32)] = t;
        holes += (int)(total & 0xffffffffull);
        movers += (int)(total >> 32);
        if (t < keep && kept) {
            mass_out[t] = mass[t];
            if (pos_out) pos_out[t] = pos[t];
        }
    }
    if (tid == 0) p.moves[bk] = holes;
    __syncthreads();
    for (int x = tid; x < holes; x += kEvictThreads) {
        mass_out[to[x]] = mass[from[x]];
        if (pos_out) pos_out[to[x]] = pos[from[x]];
    }
    for (int t = keep + tid; t < p.mass_cap; t += kEvictThreads) {
        mass_out[t] = 0.f;
        if (pos_out) pos_out[t] = -1;
    }
}

// Moves the rows; nx blocks a (sequence, key head).  A sequence whose pages were found
// shared or out of range is put back to what it was: length, weights and
// positions copied, no row moved.
__global__ void __launch_bounds__(256) streamkl_evict_move_kernel(const EvictParams p, int nx) {
    const int bk = blockIdx.x / nx, bx = blockIdx.x % nx, b = bk / p.Hk, hk = bk % p.Hk;
    if (p.refused[b] >= 0) {
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
    const int *to = p.lists + (size_t)bk * 2 * p.list, *from = to + p.list;
    const int x = threadIdx.x % (2 * ch), sub = threadIdx.x / (2 * ch);
    const PageView pv = x < ch ? p.k : p.v;
    const int *table = p.table + (size_t)b * p.table_b;
    for (int r = bx * per + sub; r < m; r += nx * per) {
        const int t = to[r], f = from[r];
        uint16_t *base = static_cast<uint16_t *>(const_cast<void *>(pv.ptr)) + hk * pv.s_head + (x % ch) * 8;
        const uint16_t *src = base + (long long)table[f / p.page] * pv.s_page + (long long)(f % p.page) * pv.s_slot;
        uint16_t *dst = base + (long long)table[t / p.page] * pv.s_page + (long long)(t % p.page) * pv.s_slot;
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
    }
}

}  // namespace skl
