// Pieces shared by the kernels of attn_fwd_paged (attn_paged.cu, attn_paged_decode.cu):
// a request's bounds, segments of work and the even split of key blocks over CTAs.
#pragma once
#include "kernels.h"
#include "ptx_sm100.cuh"

namespace gb300 {
namespace paged {

constexpr int BM = 128, BN = 128;
constexpr int kThreads = 384;
constexpr int kChunk = BM * 128;     // bytes of one 64-column chunk of a 128-row tile
constexpr float kThreshold = 8.0f;   // log2 units
constexpr int kSegs = 4;             // segment descriptors in flight

// The same value in every lane (given that it is), known to be so by the compiler.
__device__ __forceinline__ int warp_uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// Position in a ring of n slots: the slot and the parity of the pass over the ring.
template <int n>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == n) slot = 0, phase ^= 1u;
  }
};

// One segment of work, written by warp 0 and read by every other warp. It carries
// the pipeline's counters too (the warps' registers hold a row of S).
struct Seg {
  int more;       // 0: no more work
  int seq, hk;
  int q_row;      // first token's row of q and o
  int ntok;       // tokens of the unit
  int pos0;       // position of the first token among the keys (bottom-right aligned; may be negative)
  int nk;         // keys of the request
  int kt0;        // first key block
  int n0, n1;     // key blocks of tile 0 and 1 (dual: n0 in all, alternating)
  int dual;       // one tile of rows, two streams of key blocks
  int part;       // >= 0: the slot of this segment's partial O and LSE
  uint32_t v0;    // key blocks copied before this segment
  uint32_t s0, s1;  // S tiles of stream 0 and 1 before it
  uint32_t phase; // bit 0, 1: segments before it in which O_0, O_1 were written; bit 2: dual segments (all mod 2)
};
static_assert(sizeof(Seg) == 64, "OFF_SEG");

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Bounds of request s: its rows of q (clamped to the rows there are), those that are computed (the first max_q of
// them) and its keys. The causal mask aligns the last of all rows with the last key.
struct Bounds {
  int q0, n, nq, nk;
};
__device__ __forceinline__ Bounds bounds(const PagedArgs& a, int s) {
  const int c0 = __ldg(a.cu_q + s), c1 = __ldg(a.cu_q + s + 1), k = __ldg(a.seqlens_k + s);
  Bounds b;
  b.q0 = max(0, min(c0, a.total_q));
  b.n = max(0, min(c1, a.total_q) - b.q0);
  b.nq = min(b.n, a.max_q);
  b.nk = max(0, min(k, a.max_keys));
  return b;
}
// Keys that tokens up to `last` (0-based in the request) see.
__device__ __forceinline__ int keys_seen(const PagedArgs& a, const Bounds& b, int last) {
  return a.causal ? max(0, min(b.nk, last + b.nk - b.n + 1)) : b.nk;
}
// Key blocks that a unit of a request costs; a unit whose rows see no key still writes them.
__device__ __forceinline__ int unit_blocks(const PagedArgs& a, const Bounds& b, int last) {
  return max(1, ceil_div(keys_seen(a, b, last), BN));
}

// Fills a segment: tokens tok0 .. of request s, K/V head hk, key blocks [kt0, kt1).
__device__ __forceinline__ Seg make_seg(const PagedArgs& a, const Bounds& b, int s, int hk, int tok0, int ntok, int kt0,
                                        int kt1, int part) {
  Seg g;
  g.more = 1;
  g.seq = s, g.hk = hk;
  g.q_row = b.q0 + tok0;
  g.ntok = ntok;
  g.pos0 = tok0 + b.nk - b.n;
  g.nk = b.nk;
  g.kt0 = kt0;
  g.dual = ntok <= a.tile_tokens ? 1 : 0;
  g.part = part;
  const int last0 = tok0 + min(ntok, a.tile_tokens) - 1;
  g.n0 = max(0, min(ceil_div(keys_seen(a, b, last0), BN), kt1) - kt0);
  g.n1 = g.dual ? 0 : max(0, min(ceil_div(keys_seen(a, b, tok0 + ntok - 1), BN), kt1) - kt0);
  return g;
}

// The CTA of `ctas` whose range [c W / ctas, (c + 1) W / ctas) holds block x.
__device__ __forceinline__ int range_owner(long long x, long long W, int ctas) {
  const long long n = (x + 1) * ctas + W - 1;
  if (n < 0x7fffffff) return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(W)) - 1;
  return static_cast<int>(n / W) - 1;
}

// ---- even split -------------------------------------------------------------
// The key blocks of all (request, K/V head) units (one unit per pair: no request
// has more than one tile of rows), heads of a request side by side, laid end to
// end and cut into equal ranges, one per CTA.
struct EvenStart {
  int seq;           // the request that holds this CTA's first key block
  Bounds b;
  long long start;   // its first block
  long long total;   // blocks in all
  long long range0, range1;  // this CTA's
  int ctas;          // CTAs that have a range
  long long warp_sum[kThreads / 32];
};

// Called by all threads: running sums of the requests' key blocks, kThreads requests
// at a time, to the total, then a search for the request that holds this CTA's first
// block (a second pass where there are more than kThreads requests). The results are in
// *e after the caller's next __syncthreads.
__device__ __forceinline__ void even_split(const PagedArgs& a, EvenStart* e) {
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t warp = warp_id(), lane = lane_id();
  long long total = 0, range0 = 0, range1 = 0;
  int ctas = 0;
  const bool one_pass = a.num_seqs <= kThreads;
  for (int pass = 0; pass < (one_pass ? 1 : 2); ++pass) {
    long long base = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
      const int s = s0 + tid;
      int n = 0;
      Bounds b{0, 0, 0, 0};
      if (s < a.num_seqs) {
        b = bounds(a, s);
        n = b.nq > 0 ? unit_blocks(a, b, b.nq - 1) : 0;
      }
      long long inc = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, d);
        if (static_cast<int>(lane) >= d) inc += u;
      }
      if (lane == 31) e->warp_sum[warp] = inc;
      __syncthreads();
      long long before = base, all = base;
#pragma unroll
      for (uint32_t w = 0; w < kThreads / 32; ++w) {
        const long long x = e->warp_sum[w];
        if (w < warp) before += x;
        all += x;
      }
      if (one_pass || (pass == 0 && s0 + kThreads >= a.num_seqs)) {
        total = all * a.heads_kv;
        // at least kPagedMinBlocks key blocks per CTA: fewer would cost more to merge than they save
        const long long want = (total + kPagedMinBlocks - 1) / kPagedMinBlocks;
        ctas = static_cast<int>(want < static_cast<long long>(gridDim.x) ? want : gridDim.x);
        const int c = static_cast<int>(blockIdx.x);
        if (c < ctas) {
          if (total < (1 << 23)) {  // 32-bit products (ctas <= 152): a 64-bit division takes hundreds of cycles
            range0 = static_cast<uint32_t>(c) * static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas);
            range1 = static_cast<uint32_t>(c + 1) * static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas);
          } else {
            range0 = c * total / ctas;
            range1 = (c + 1) * total / ctas;
          }
        }
      }
      const long long start = (before + inc - n) * a.heads_kv;
      if ((one_pass || pass == 1) && n > 0 && start <= range0 &&
          range0 < start + static_cast<long long>(n) * a.heads_kv) {
        e->seq = s;
        e->b = b;
        e->start = start;
      }
      base = all;
      if (!one_pass) __syncthreads();
    }
  }
  if (tid == 0) {
    e->total = total;
    e->range0 = range0, e->range1 = range1;
    e->ctas = ctas;
  }
}

// Walks this CTA's range, one segment (a unit's part in the range) after another;
// run by one warp, all lanes alike.
struct EvenWalk {
  int s = 0, hk = 0, kt = 0, unit = 0;
  Bounds b{0, 0, 0, 0}, b_next{0, 0, 0, 0};  // request s and, fetched ahead, s + 1
  long long g = 0, range1 = 0;
  bool merged = false;  // a unit begins in this range and ends beyond it: at most one

  __device__ __forceinline__ void fetch_next(const PagedArgs& a) {
    if (s + 1 < a.num_seqs) b_next = bounds(a, s + 1);
  }
  __device__ __forceinline__ void begin(const PagedArgs& a, const EvenStart* e) {
    g = e->range0, range1 = e->range1;
    if (g >= range1) return;
    s = e->seq;
    b = e->b;
    unit = unit_blocks(a, b, b.nq - 1);
    fetch_next(a);
    const long long off = g - e->start;
    hk = off < 0x7fffffff ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(unit))
                          : static_cast<int>(off / unit);
    kt = static_cast<int>(off - static_cast<long long>(hk) * unit);
  }
  __device__ __forceinline__ Seg next(const PagedArgs& a, const EvenStart* e) {
    Seg w;
    w.more = 0, w.n0 = w.n1 = 0;
    if (g >= range1) return w;
    const int take = static_cast<int>(min(static_cast<long long>(unit - kt), range1 - g));
    int part = -1;
    if (kt > 0) part = static_cast<int>(blockIdx.x);                     // continues an earlier CTA's unit
    else if (take < unit) part = static_cast<int>(gridDim.x + blockIdx.x);  // begins here, ends beyond
    w = make_seg(a, b, s, hk, 0, b.nq, kt, kt + take, part);
    if (kt == 0 && take < unit) {
      merged = true;
      if (lane_id() == 0) {
        MergeUnit m;
        m.q_row = w.q_row, m.ntok = w.ntok, m.hk = hk;
        m.first = part;
        m.rest = static_cast<int>(blockIdx.x) + 1;
        m.n = range_owner(g + unit - 1, e->total, e->ctas) - static_cast<int>(blockIdx.x) + 1;
        a.merge[blockIdx.x] = m;
      }
    }
    g += take;
    kt = 0;
    if (g < range1 && ++hk == a.heads_kv) {  // (the unit ended, or the range did)
      hk = 0;
      do {
        b = b_next, ++s;
        fetch_next(a);
      } while (b.nq == 0 && s + 1 < a.num_seqs);
      unit = unit_blocks(a, b, b.nq - 1);
    }
    return w;
  }
  // At the end of the range: no unit to merge begins here.
  __device__ __forceinline__ void finish(const PagedArgs& a) const {
    if (!merged && lane_id() == 0) a.merge[blockIdx.x].n = 0;
  }
};

// The page of key block kt that lane's box number my_page of a block's copies reads;
// num_pages (whose boxes read zeros) past the last key and for entries outside the cache.
// (Positions fit in 31 bits: max_keys.)
__device__ __forceinline__ int page_of(const PagedArgs& a, const int* table, int nk, int kt, int my_page) {
  const int key = (kt << 7) + (my_page << a.page_shift);
  if (key >= nk) return a.num_pages;
  const uint32_t pg = static_cast<uint32_t>(__ldg(table + (key >> a.page_shift)));
  return static_cast<int>(min(pg, static_cast<uint32_t>(a.num_pages)));
}

// Warp 0 of both kernels: publishes the segments that next_seg() gives and copies their K
// and V blocks (and, by copy_q(w), Q) into the rings, one box per page and 64 columns, each
// lane issuing one. K runs up to two blocks ahead of V, which is needed only a softmax
// later: a K block that waited behind a V slot left the tensor cores idle for a copy's
// latency (chunks of 24 requests: 604 us so, 4,080 cycles per pair of blocks where the
// products take 2,048). The next segment and its first page are looked up behind the
// first few copies. Returns false when a wait ran out; the copies in flight have landed then.
template <typename C, typename B, typename NextSeg, typename CopyQ>
__device__ __forceinline__ bool copy_loop(const PagedArgs& a, B* bar, Seg* sSeg, uint8_t* sK, uint8_t* sV,
                                          const CUtensorMap* tmk, const CUtensorMap* tmv, uint32_t site,
                                          NextSeg&& next_seg, CopyQ&& copy_q) {
  const int lane = static_cast<int>(lane_id());
  const int np = a.page_size < BN ? BN >> a.page_shift : 1;  // pages (boxes along the keys) of a key block
  const int box_rows = a.page_size < BN ? a.page_size : BN;
  const int my_page = lane % np, my_chunk = lane / np;
  const uint32_t box_off = my_chunk * kChunk + my_page * box_rows * 128;
  Ring<C::NK> rk;
  Ring<C::NV> rv;
  Ring<kSegs> rs;
  uint32_t done = 0;  // key blocks of the segments so far
  uint32_t cs0 = 0, cs1 = 0, phase = 0;
  int jk = 0, jv = 0;
  bool ok = true;
  Seg w, nw;          // this segment and the next
  const int* table;   // block-table rows of both
  const int* ntable = nullptr;
  int npage = 0;
  nw.more = 1;
  bool first = true;
  for (;;) {
    // the next segment and its first page; at the start, then behind each segment's first few copies
    auto look_ahead = [&]() {
      nw = next_seg();
      if (nw.more) {
        ntable = a.block_table + nw.seq * a.block_table_stride;
        npage = page_of(a, ntable, nw.nk, nw.kt0, my_page);
      }
    };
    int n = 0;
    if (!first) {
      w = nw;
      table = ntable;
      ok = mbar_wait_warp(&bar->seg_empty[rs.slot], rs.phase ^ 1u, a.status, site);
      if (!ok) break;
      n = max(w.n0, w.n1);
      if (lane == 0) {
        w.v0 = done, w.s0 = cs0, w.s1 = cs1, w.phase = phase;
        sSeg[rs.slot] = w;
        mbar_arrive(&bar->seg_full[rs.slot]);
      }
      rs.next();
      if (!w.more) break;
      cs0 += w.dual ? (w.n0 + 1) / 2 : w.n0;
      cs1 += w.dual ? w.n0 / 2 : w.n1;
      phase ^= (w.n0 > 0 ? 1u : 0u) | ((w.dual ? w.n0 > 1 : w.n1 > 0) ? 2u : 0u) | (w.dual ? 4u : 0u);
    }
    first = false;
    int kp = npage, p1 = 0, p2 = 0;  // pages of K block jk, jk - 1 and jk - 2
    const int ahead = min(n, static_cast<int>(C::NK));
    bool looked = false;
    for (jk = jv = 0;;) {
      if (jk >= ahead && !looked) {
        look_ahead();
        looked = true;
      }
      if (jv >= n) break;
      const bool is_k = jk < n && jk - jv < 2;
      if (is_k) {
        const int next = jk + 1 < n ? page_of(a, table, w.nk, w.kt0 + jk + 1, my_page) : 0;  // fetched ahead of the wait
        ok = mbar_wait_warp(&bar->k_empty[rk.slot], rk.phase ^ 1u, a.status, site + 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar->k_full[rk.slot], C::K_BYTES);
        __syncwarp();
        const int row = a.page_size > BN ? ((w.kt0 + jk) << 7) & (a.page_size - 1) : 0;
        if (my_chunk < C::QCH)
          tma_load_4d(sK + rk.slot * C::K_BYTES + box_off, tmk, &bar->k_full[rk.slot], my_chunk * 64, w.hk, row, kp);
        rk.next();
        p2 = p1, p1 = kp, kp = next;
        if (++jk == 1) {  // Q behind the first K: that slot may be free long before the previous Q is
          ok = copy_q(w);
          if (!ok) break;
        }
      } else {
        ok = mbar_wait_warp(&bar->v_empty[rv.slot], rv.phase ^ 1u, a.status, site + 2);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar->v_full[rv.slot], C::V_BYTES);
        __syncwarp();
        const int row = a.page_size > BN ? ((w.kt0 + jv) << 7) & (a.page_size - 1) : 0;
        if (my_chunk < C::VCH)
          tma_load_4d(sV + rv.slot * C::V_BYTES + box_off, tmv, &bar->v_full[rv.slot], my_chunk * 64, w.hk, row,
                      jk - jv == 2 ? p2 : p1);
        rv.next();
        ++jv;
      }
    }
    if (!ok) break;
    done += static_cast<uint32_t>(n);
  }
  if (!ok) {
    const uint32_t ck = done + static_cast<uint32_t>(jk), cv = done + static_cast<uint32_t>(jv);
    for (uint32_t u = 0; u < C::NK && u < ck; ++u)
      mbar_wait(&bar->k_full[(ck - 1 - u) % C::NK], ((ck - 1 - u) / C::NK) & 1u, nullptr, 0);
    for (uint32_t u = 0; u < C::NV && u < cv; ++u)
      mbar_wait(&bar->v_full[(cv - 1 - u) % C::NV], ((cv - 1 - u) / C::NV) & 1u, nullptr, 0);
  }
  return ok;
}

}  // namespace paged
}  // namespace gb300
