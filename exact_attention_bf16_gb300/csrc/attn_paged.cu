// Attention of packed new tokens over a paged KV cache (attn_fwd_paged).
//
// O_i = sum_j softmax_j(a_ij) v_j over the visible keys of query i, a_ij =
// scale q_i . k_j, in one pass over the keys with a running maximum m and sum l
// (log2 units) per row, the conditional rescale of fwd_kernel.cuh (a row's m is
// replaced only when a block exceeds it by more than 8) and O accumulated in
// Tensor Memory.
//
// Rows. The query heads of one K/V head share its keys, so the rows of a tile
// are (token, head of the group) pairs, token-major: a 128-row tile holds
// 128 / group tokens, and K/V are read once for the whole group. A unit of work
// is up to 256 such rows (two tiles, each with its own S and O) of one request
// and K/V head, or up to 128 rows, which then run as two streams over the even
// and the odd key blocks (one computes S while the other's softmax runs), merged
// at the end: a decoding request has few rows and many keys, and one stream's
// chain S -> softmax -> PV would leave the copies waiting.
//
// Splitting. A unit's key blocks may be cut into segments taken by different
// CTAs; each writes its normalised fp32 O and its LSE (log2), and
// merge_kernel adds them with the weights 2^(LSE_r - LSE), in key order.
// One persistent CTA per SM (shared memory and Tensor Memory are taken whole):
//   - up to 128 rows per request (a few proposed tokens; up to 16 rows without a score
//     modification run in attn_paged_decode.cu instead): bound by
//     HBM (every K/V byte is read once and used for a handful of rows), so the
//     key blocks of all (request, K/V head) units, laid end to end, are cut into
//     equal ranges, one per CTA. A CTA finds its range from the lengths alone. 33 requests
//     of 3..6 tokens, 16 heads over 1, d = 64, up to 16384 keys: 26.4 us (about five key
//     blocks a CTA), 28 by the list below; 64 decoding requests 321 us against 393.
//   - longer chunks: bound by the tensor cores, and by L2 where concurrent CTAs
//     read different keys, so units are taken one after another from a list
//     that chunk_list_kernel builds, a request's units together, long requests
//     and late units (the most keys under the causal mask) first. Only units
//     longer than an equal share of the work are cut. 24 requests, chunks of 500..2048 tokens over
//     up to 16384 keys, 32 heads over 8, d = 128: 512 us, 1190 TFLOP/s; four times the work over
//     like lengths 1360 (the contiguous causal forward: 1230 at 4096 keys, 1450 at 8192, 1590 at 32768). The tensor
//     pipe is active 55% of the time. A pair of blocks takes some 3,760 cycles: the chain S -> softmax -> PV of the two
//     tiles 2,900, the rest is the units' ends, single tokens that share the list, the list itself and the merge.
//
// Warps: 0 work and TMA copies, 1 MMA issue, 4..7 and 8..11 softmax of tile or
// stream 0 and 1. K and V have rings of their own; a copy is one box per page
// and 64 columns, each lane of warp 0 issuing one. Pages past a request's last
// key and entries outside the cache become a page index past the cache, whose
// boxes read zeros.
//
// P enters the PV product in bf16, V's type in the cache (half a step is 2^-8 of
// each weight): an fp16 copy of V, as the contiguous forward makes, would cost a
// second pass over keys that a decoding step reads only once. Every sum is fp32.
#include <cstddef>
#include <type_traits>

#include "kernels.h"
#include "paged_common.cuh"
#include "ptx_sm100.cuh"
#include "score_mod.cuh"

namespace gb300 {
namespace paged {

__host__ __device__ constexpr uint32_t tS(int i) { return 128u * i; }
__host__ __device__ constexpr uint32_t tO(int i) { return 256u + 128u * i; }

// The even split has one tile of rows, so its shared memory holds more of K and V.
template <int DQK, int DV, bool EVEN>
struct Cfg {
  static constexpr int QT = EVEN ? 1 : 2;
  static constexpr int QCH = DQK / 64, VCH = DV / 64;
  static constexpr int Q_BYTES = QCH * kChunk;
  static constexpr int K_BYTES = QCH * kChunk;
  static constexpr int V_BYTES = VCH * kChunk;
  // ring slots: what shared memory holds beside the Q tiles
  static constexpr int NK = DQK == 64 ? 6 : (DQK == 128 ? 3 : 2);
  static constexpr int NV = DQK == 64 ? 6 : (EVEN ? (DQK == 128 ? 3 : 2) : (DQK == 128 ? 2 : 1));
  static constexpr int OFF_K = QT * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * K_BYTES;
  static constexpr int OFF_X = OFF_V + NV * V_BYTES;  // the streams' (m, l): [2 streams][128] float2
  static constexpr int OFF_SEG = OFF_X + 2 * BM * 8;
  static constexpr int OFF_BAR = OFF_SEG + kSegs * 64;
  static constexpr int SMEM = OFF_BAR + 640;  // the base is 1024-byte aligned (checked)
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr uint32_t REG_LO = 96, REG_HI = 200;
  static constexpr int REG_BUDGET = 128 * REG_LO + 256 * REG_HI;
};

struct Bars {
  // one arrival
  uint64_t q_full, q_free;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], o_full[2];
  uint64_t seg_full[kSegs];
  uint64_t mma_done;
  // four: a warpgroup's warps
  uint64_t p_full[2];
  uint64_t x_full[2];  // dual: a stream's (m, l) are in shared memory
  // nine: eight softmax warps and the MMA thread
  uint64_t seg_empty[kSegs];
  uint64_t o_free;     // a segment is over: its O has been read, its MMAs issued (so neither side gets two ahead)
  uint32_t tmem_base;
  EvenStart even;
};
static_assert(sizeof(Bars) <= 640, "barriers must fit their reserved bytes");

// EVEN: the even split of all units' key blocks (at most one tile of rows per
// request); else the list of chunk_list_kernel.
template <int DQK, int DV, int MOD, bool EVEN>
__global__ void __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, const PagedArgs a) {
  using C = Cfg<DQK, DV, EVEN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {  // the 128-byte-swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(a.status, DEV_BAD_CONFIG, 0x3000);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  float2* sX = reinterpret_cast<float2*>(smem + C::OFF_X);
  Seg* sSeg = reinterpret_cast<Seg*>(smem + C::OFF_SEG);
  Bars* bar = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const uint32_t warp = warp_id(), lane = lane_id();

  constexpr int kOnes = offsetof(Bars, p_full) / 8, kFours = offsetof(Bars, seg_empty) / 8,
                kAll = offsetof(Bars, tmem_base) / 8;
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kAll) {  // one thread per barrier
    const int x = static_cast<int>(threadIdx.x) - 64;
    mbar_init(reinterpret_cast<uint64_t*>(bar) + x, x < kOnes ? 1 : x < kFours ? 4 : 9);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
  }
  if constexpr (EVEN) even_split(a, &bar->even);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bar->tmem_base;
  // merge_kernel may be launched (its blocks fit only as these CTAs leave), and this kernel's own
  // reads of chunk_list_kernel's list begin
  if constexpr (!EVEN) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < 4) {
    regs_dec<C::REG_LO>();
    if (warp == 0) {
      // ===================== work and copies ================================
      const uint32_t q_bytes = static_cast<uint32_t>(a.kv_group * a.tile_tokens) * 128u * C::QCH;
      uint32_t cq = 0;
      EvenWalk walk;
      if constexpr (EVEN) walk.begin(a, &bar->even);
      int item = static_cast<int>(blockIdx.x);  // list: this CTA's next entry
      const int n_items = EVEN ? 0 : a.list->n_items, n_parts = EVEN ? 0 : a.list->n_parts;
      const int first_unit = 2 * static_cast<int>(gridDim.x);
      const bool ok = copy_loop<C>(
          a, bar, sSeg, sK, sV, &tmk, &tmv, 0x3100,
          [&]() -> Seg {
            if constexpr (EVEN) {
              return walk.next(a, &bar->even);
            } else {
              Seg w;
              w.more = 0, w.n0 = w.n1 = 0;
              while (item < n_items) {
                const ChunkItem it = a.items[item < n_parts ? item : item - n_parts + first_unit];
                int nx = 0;
                if (lane == 0) nx = atomicAdd(&a.list->next, 1);  // needed one segment later
                item = __shfl_sync(0xffffffffu, nx, 0);
                if (it.seq < 0) continue;  // a unit that was cut: its parts are entries of their own
                const Bounds b = bounds(a, it.seq);
                w = make_seg(a, b, it.seq, it.hk, it.tok0, min(b.nq - it.tok0, 2 * a.tile_tokens), it.kt0, it.kt1, it.part);
                break;
              }
              return w;
            }
          },
          [&](const Seg& w) {
            if (!mbar_wait_warp(&bar->q_free, (cq & 1u) ^ 1u, a.status, 0x3120)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&bar->q_full, q_bytes * (w.dual ? 1u : 2u));
            __syncwarp();
            const int tiles = w.dual ? 1 : 2;
            if (static_cast<int>(lane) < tiles * C::QCH) {
              const int t = static_cast<int>(lane) / C::QCH, c = static_cast<int>(lane) % C::QCH;
              tma_load_4d(sQ + t * C::Q_BYTES + c * kChunk, &tmq, &bar->q_full, c * 64, w.hk * a.kv_group,
                          w.q_row + t * a.tile_tokens, 0);
            }
            ++cq;
            return true;
          });
      if constexpr (EVEN) walk.finish(a);
      if (!ok && cq > 0) mbar_wait(&bar->q_full, (cq - 1) & 1u, nullptr, 0);
    } else if (warp == 1) {
      // ===================== MMA issue ======================================
      // The whole warp walks the loop, so that its counters and descriptors are uniform across it; lane 0 issues.
      constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false, false);
      constexpr uint32_t idO = idesc_bf16_f32(BM, DV, false, true);
      Ring<C::NK> rk;
      Ring<C::NV> rv;
      uint32_t cq = 0, seg_i = 0, pp = 0;  // pp: a bit per stream
      bool ok = true;
      const uint64_t dq0 = smem_desc(smem_u32(sQ), 16, 1024, SWZ_128B), dk0 = smem_desc(smem_u32(sK), 16, 1024, SWZ_128B);
      const uint64_t dv0 = smem_desc(smem_u32(sV), kChunk, 1024, SWZ_128B);
      // A commit costs the issuing thread several hundred cycles, so K and V slots are released by the
      // softmax warps: S of block j follows PV of the block before on its stream in issue order. (With one V
      // slot the last block would wait for a release that follows it: that ring is released by commits.)
      auto issue_s = [&](int i, int q_tile) {
        const uint64_t dq = desc_add(dq0, q_tile * C::Q_BYTES), dk = desc_add(dk0, rk.slot * C::K_BYTES);
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk) {
            const uint32_t off = (kk / 4) * kChunk + (kk % 4) * 32;
            mma_ss(tbase + tS(i), desc_add(dq, off), desc_add(dk, off), idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bar->s_full[i]);
        }
      };
      auto issue_pv = [&](int i, bool first) {
        const uint64_t dv = desc_add(dv0, rv.slot * C::V_BYTES);
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tbase + tO(i), tbase + tS(i) + kk * 8, desc_add(dv, kk * 2048), idO, (kk > 0 || !first) ? 1u : 0u);
        }
      };
      auto v_done = [&]() {
        if (C::NV == 1 && lane == 0) mma_commit(&bar->v_empty[rv.slot]);
        rv.next();
      };
      for (;;) {
        const int slot = static_cast<int>(seg_i % kSegs);
        ok = mbar_wait_warp(&bar->seg_full[slot], (seg_i / kSegs) & 1u, a.status, 0x3200);
        if (!ok) break;
        const Seg* w = sSeg + slot;
        const int more = warp_uniform(w->more), n0 = warp_uniform(w->n0), n1 = warp_uniform(w->n1);
        const bool dual = EVEN || warp_uniform(w->dual) != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->seg_empty[slot]);
        if (!more) break;
        const int n = max(n0, n1);
        // the previous segment's O has been read: before the first PV overwrites it
        auto wait_o = [&]() { return seg_i == 0 || mbar_wait_warp(&bar->o_free, (seg_i - 1) & 1u, a.status, 0x3210); };
        if (n == 0) ok = wait_o();
        for (int j = 0; j <= n && n > 0 && ok; ++j) {
          if (dual) {
            if (j < n) {
              ok = mbar_wait_warp(&bar->k_full[rk.slot], rk.phase, a.status, 0x3220);
              if (ok && j == 0) ok = mbar_wait_warp(&bar->q_full, cq & 1u, a.status, 0x3230);
              if (!ok) break;
              tc_fence_after();
              issue_s(j & 1, 0);
              rk.next();
              if (j == n - 1 && lane == 0) mma_commit(&bar->q_free);
            }
            if (j > 0) {
              const int i = (j - 1) & 1;
              if (j == 1) ok = wait_o();
              ok = ok && mbar_wait_warp(&bar->v_full[rv.slot], rv.phase, a.status, 0x3240) &&
                   mbar_wait_warp(&bar->p_full[i], (pp >> i) & 1u, a.status, 0x3250);
              if (!ok) break;
              tc_fence_after();
              pp ^= 1u << i;
              issue_pv(i, j <= 2);
              v_done();
              if (j - 1 >= n - 2 && lane == 0) mma_commit(&bar->o_full[i]);
            }
          } else {
            // What the step's first products need is tested together: this warp's instructions are the step's limit, and
            // waits one after another cost 150 to 400 cycles each even where everything had arrived.
            const bool pv0 = j > 0 && j - 1 < n0;
            const bool k_in = j == n || mbar_test(&bar->k_full[rk.slot], rk.phase);
            const bool v_in = j == 0 || mbar_test(&bar->v_full[rv.slot], rv.phase);
            const bool p_in = !pv0 || mbar_test(&bar->p_full[0], pp & 1u);
            if (j < 2 || !__all_sync(0xffffffffu, k_in && v_in && p_in)) {
              ok = (j == n || mbar_wait_warp(&bar->k_full[rk.slot], rk.phase, a.status, 0x3220)) &&
                   (j != 0 || mbar_wait_warp(&bar->q_full, cq & 1u, a.status, 0x3230)) && (j != 1 || wait_o()) &&
                   (j == 0 || mbar_wait_warp(&bar->v_full[rv.slot], rv.phase, a.status, 0x3240)) &&
                   (!pv0 || mbar_wait_warp(&bar->p_full[0], pp & 1u, a.status, 0x3250));
              if (!ok) break;
            }
            tc_fence_after();
#pragma unroll 1  // (unrolled 552 us, so 512: the code no longer fits what the instruction caches keep for this warp)
            for (int i = 0; i < 2; ++i) {
              const int ni = i == 0 ? n0 : n1;
              if (j > 0 && j - 1 < ni) {
                if (i == 1) {
                  ok = mbar_wait_warp(&bar->p_full[1], (pp >> 1) & 1u, a.status, 0x3251);
                  if (!ok) break;
                  tc_fence_after();
                }
                pp ^= 1u << i;
                issue_pv(i, j == 1);
                if (j == ni && lane == 0) mma_commit(&bar->o_full[i]);
              }
              if (j < ni) issue_s(i, i);
            }
            if (!ok) break;
            if (j > 0) v_done();
            if (j < n) {
              rk.next();
              if (j == n - 1 && lane == 0) mma_commit(&bar->q_free);
            }
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bar->o_free);
        if (n > 0) ++cq;
        ++seg_i;
      }
      if (lane == 0) {
        mma_commit(&bar->mma_done);
        mbar_wait(&bar->mma_done, 0, a.status, 0x32ff);
      }
    }
  } else {
    regs_inc<C::REG_HI>();
    // ======================= softmax and output =============================
    const int i = (static_cast<int>(warp) - 4) / 4;  // tile or stream
    const uint32_t quarter = warp & 3u;
    const uint32_t lane_base = tbase + ((quarter * 32u) << 16);
    // This thread's row of a segment: token and head of the group (divided anew where needed).
    auto row_tok = [&](int dual) {
      const int r = static_cast<int>(quarter * 32 + lane);
      return r / a.kv_group + (EVEN || dual ? 0 : i * a.tile_tokens);
    };
    auto row_valid = [&](const volatile Seg& w) {
      const int r = static_cast<int>(quarter * 32 + lane);
      return r < a.kv_group * a.tile_tokens && row_tok(EVEN || w.dual) < w.ntok;
    };
    bool ok = true;
    for (uint32_t seg_i = 0;; ++seg_i) {
      // read where needed (volatile: not kept in registers across the blocks' loop)
      const volatile Seg& w = sSeg[seg_i % kSegs];
      ok = mbar_wait_warp(&bar->seg_full[seg_i % kSegs], (seg_i / kSegs) & 1u, a.status, 0x3300);
      if (!ok || !w.more) break;
      float m_used = -INFINITY, l = 0.f;
      {
        const bool valid = row_valid(w);
        const int pos = w.pos0 + row_tok(w.dual);  // the row's position among the keys
        // (rows without a token hold whatever shared memory did: computed without masks, never stored)
        const int klim = !valid ? 0x7fffffff : (a.causal ? max(0, min(w.nk, pos + 1)) : w.nk);
        const bool work = __any_sync(0xffffffffu, valid);  // a warp without rows only keeps the barriers in step
        float slope = 0.f;
        if (MOD == kModAlibi && valid)
          slope = fabsf(__ldg(a.alibi_slopes + w.hk * a.kv_group + static_cast<int>(quarter * 32 + lane) % a.kv_group) *
                        a.inv_scale);
        // whether this lane's page of key block kt holds keys (one lane per page of a block)
        auto page_ok = [&](int kt) -> bool {
          const int np = a.page_size < BN ? BN >> a.page_shift : 1;
          const long long key = (static_cast<long long>(kt) << 7) + (static_cast<long long>(lane) << a.page_shift);
          if (static_cast<int>(lane) >= np || key >= w.nk) return true;
          const int pg = __ldg(a.block_table + w.seq * a.block_table_stride + (key >> a.page_shift));
          return pg >= 0 && pg < a.num_pages;
        };
        const int step = EVEN || w.dual ? 2 : 1;
        int kt = w.kt0 + (EVEN || w.dual ? i : 0);
        const int kt_end = w.kt0 + (EVEN || w.dual || i == 0 ? w.n0 : w.n1);
        uint32_t s_phase = i == 0 ? w.s0 : w.s1;
        bool first = true;
        bool pg_ok = kt < kt_end ? page_ok(kt) : true;
        for (; kt < kt_end; kt += step, ++s_phase, first = false) {
          const uint32_t pages = __ballot_sync(0xffffffffu, pg_ok);
          if (kt + step < kt_end) pg_ok = page_ok(kt + step);  // fetched one block ahead
          ok = mbar_wait_warp(&bar->s_full[i], s_phase & 1u, a.status, 0x3310 + i);
          if (!ok) break;
          // K of this block has been read, and V of the stream's block before (not dual: by tile 1's S, which is
          // the last of the block's and tile 1 has every block that tile 0 has)
          if (quarter == 0 && lane == 0 && (EVEN || w.dual || i == 1)) {
            const uint32_t u = w.v0 + static_cast<uint32_t>(kt - w.kt0);
            mbar_arrive(&bar->k_empty[u % C::NK]);
            if (C::NV > 1 && !first) mbar_arrive(&bar->v_empty[(u - step) % C::NV]);
          }
          tc_fence_after();
          if (work) {
            uint32_t s[BN];
            tmem_ld32(lane_base + tS(i) + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
            tmem_ld32(lane_base + tS(i) + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
            tmem_ld32(lane_base + tS(i) + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
            tmem_ld32(lane_base + tS(i) + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
            tmem_wait_ld();
            if constexpr (MOD == kModSoftcap) {
#pragma unroll
              for (int c = 0; c < BN; ++c) s[c] = __float_as_uint(a.mod_b * tanh_scaled(__uint_as_float(s[c]), a.mod_k2));
            } else if constexpr (MOD == kModAlibi) {
              const float base = slope * static_cast<float>(kt * BN - pos);
#pragma unroll
              for (int c = 0; c < BN; ++c)
                s[c] = __float_as_uint(__uint_as_float(s[c]) - fabsf(fmaf(slope, static_cast<float>(c), base)));
            }
            const int cnt = klim - kt * BN;  // visible keys of this row in the block
            if (cnt < BN) {
#pragma unroll
              for (int c = 0; c < BN; ++c)
                if (c >= cnt) s[c] = __float_as_uint(-INFINITY);
            }
            if (pages != 0xffffffffu) {  // keys on pages outside the cache (warp-uniform branch)
              const int sh = a.page_size < BN ? a.page_shift : 7;
#pragma unroll
              for (int c = 0; c < BN; c += 16)
                if (!((pages >> (c >> sh)) & 1u)) {
#pragma unroll
                  for (int u = 0; u < 16; ++u) s[c + u] = __float_as_uint(-INFINITY);
                }
            }
            float mp[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) mp[c] = fmaxf(__uint_as_float(s[c]), __uint_as_float(s[c + 8]));
#pragma unroll
            for (int c = 16; c < BN; c += 16)
#pragma unroll
              for (int z = 0; z < 8; ++z) mp[z] = fmax3(mp[z], __uint_as_float(s[c + z]), __uint_as_float(s[c + 8 + z]));
            const float mx = fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
            const float sl2 = a.scale_log2;
            const float m_tile = mx * sl2;
            const bool need = valid && m_tile > m_used + kThreshold;
            float alpha = 1.f;
            if (need) {
              alpha = (m_used == -INFINITY) ? 0.f : ex2_mufu(m_used - m_tile);
              m_used = m_tile;
            }
            l *= alpha;
            const float mu = (m_used == -INFINITY) ? 0.f : m_used;
            uint32_t pk[BN / 2];
            float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 sl2v = make_float2(sl2, sl2), negmu = make_float2(-mu, -mu);
#pragma unroll
            for (int c = 0; c < BN / 2; ++c) {
              const float2 x = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2v, negmu);
              const float2 p = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
              pk[c] = pack_bf16x2(p.x, p.y);
              rs[c & 1] = fadd2(rs[c & 1], p);
            }
            l += (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
            tmem_st32(lane_base + tS(i) + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
            tmem_st32(lane_base + tS(i) + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
            if (!first && __any_sync(0xffffffffu, need)) {
#pragma unroll
              for (int c = 0; c < DV / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(lane_base + tO(i) + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 32; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * alpha);
                tmem_st32(lane_base + tO(i) + c * 32, o);
              }
            }
          }
          // The request's last block: cache rows past its last key, on the page that holds it, may be
          // anything (0 x NaN is NaN), so they are zeroed before the PV product reads them. Tile 0's
          // warps do it where it has this block: its PV comes first and waits for them.
          const int tail = w.nk - kt * BN;  // keys of the request in this block
          if (tail < BN && tail > 0 && (tail & (a.page_size - 1)) != 0 && (w.dual || i == 0 || kt >= w.kt0 + w.n0)) {
            const uint32_t u = w.v0 + static_cast<uint32_t>(kt - w.kt0), vs = u % C::NV;
            // one slot: the block before may not have been read yet, and its phase of v_full not have come
            if (C::NV == 1 && u > 0) ok = mbar_wait_warp(&bar->v_empty[0], (u - 1) & 1u, a.status, 0x3321);
            ok = ok && mbar_wait_warp(&bar->v_full[vs], (u / C::NV) & 1u, a.status, 0x3320);
            if (!ok) break;
            const int end = min(BN, (tail | (a.page_size - 1)) + 1);
            uint8_t* v = sV + vs * C::V_BYTES;
            const int units = (end - tail) * 8;  // 16-byte pieces of a chunk
            for (int x = static_cast<int>(quarter * 32 + lane); x < units * C::VCH; x += 128)
              *reinterpret_cast<uint4*>(v + (x / units) * kChunk + tail * 128 + (x % units) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->p_full[i]);
        }
      }
      if (!ok) break;
      // ---- output
      const bool dual = EVEN || w.dual != 0;
      const bool has0 = (dual || i == 0 ? w.n0 : w.n1) > 0;  // O_0 (dual) or this tile's O was written
      const bool has1 = dual && w.n0 > 1;
      // every warp has left the segment before (its reads of sX among them)
      if (seg_i > 0) ok = mbar_wait_warp(&bar->o_free, (seg_i - 1) & 1u, a.status, 0x3328);
      if (!ok) break;
      const int r = static_cast<int>(quarter * 32 + lane);
      float lse2;      // the row's LSE in log2 units
      // Weights of O_0 (or this tile's O) and, dual, of O_1; kNoKeys where the row saw no key: nothing is added then, also
      // beside values that are not finite (0 x NaN). (A flag beside each weight cost the chunks spills and 3%.)
      constexpr float kNoKeys = -0.f;
      float w0, w1 = kNoKeys;
      if (dual) {
        sX[i * BM + r] = make_float2(m_used, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->x_full[i]);
        ok = mbar_wait_warp(&bar->x_full[1 - i], (w.phase >> 2) & 1u, a.status, 0x3330);
        if (!ok) break;
        const float2 y = sX[(1 - i) * BM + r];
        const float ma = i == 0 ? m_used : y.x, la = i == 0 ? l : y.y, mb = i == 0 ? y.x : m_used, lb = i == 0 ? y.y : l;
        const float mm = fmaxf(ma, mb);
        // (a sum of 0 is a row without keys; a NaN sum is no such row, and stays NaN in O and LSE)
        const float ea = la != 0.f ? ex2_mufu(ma - mm) : 0.f, eb = lb != 0.f ? ex2_mufu(mb - mm) : 0.f;
        const float lt = la * ea + lb * eb;
        const float inv_l = lt != 0.f ? 1.f / lt : 0.f;
        lse2 = lt != 0.f ? mm + log2f(lt) : -INFINITY;
        w0 = la != 0.f ? ea * inv_l : kNoKeys, w1 = lb != 0.f ? eb * inv_l : kNoKeys;
        // (the exchange above also says that the other warpgroup has left the segment before, so
        // that its O barrier is at most one phase behind)
        if (has0) ok = mbar_wait_warp(&bar->o_full[0], w.phase & 1u, a.status, 0x3340);
        if (ok && has1) ok = mbar_wait_warp(&bar->o_full[1], (w.phase >> 1) & 1u, a.status, 0x3341);
      } else {
        w0 = l != 0.f ? 1.f / l : kNoKeys;
        lse2 = l != 0.f ? m_used + log2f(l) : -INFINITY;
        if (has0) ok = mbar_wait_warp(&bar->o_full[i], (w.phase >> i) & 1u, a.status, 0x3340 + i);
      }
      if (!ok) break;
      if (C::NV > 1 && quarter == 0 && lane == 0 && i == (dual ? 0 : 1)) {  // the last V blocks
        const uint32_t end = w.v0 + static_cast<uint32_t>(dual ? w.n0 : w.n1);
        if (has1) mbar_arrive(&bar->v_empty[(end - 2) % C::NV]);
        if (has0) mbar_arrive(&bar->v_empty[(end - 1) % C::NV]);
      }
      tc_fence_after();
      const int tok = row_tok(dual), head = w.hk * a.kv_group + r % a.kv_group, part = w.part;
      const bool valid = row_valid(w);
      if (__any_sync(0xffffffffu, valid)) {
        const int c_lo = dual ? i * (DV / 64) : 0, c_hi = dual ? (i + 1) * (DV / 64) : DV / 32;  // 32-column groups
        const int64_t prow = static_cast<int64_t>(part) * a.part_rows + (dual ? 0 : i * BM) + r;
        __nv_bfloat16* orow = a.o + static_cast<int64_t>(w.q_row + tok) * a.o_row + static_cast<int64_t>(head) * a.o_head;
        auto keys = [](float weight) { return __float_as_uint(weight) != __float_as_uint(kNoKeys); };
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t o[32];  // (columns never written are read too, but not used)
          tmem_ld32(lane_base + (dual ? tO(0) : tO(i)) + c * 32, o);
          if (dual) {
            uint32_t o1[32];
            tmem_ld32(lane_base + tO(1) + c * 32, o1);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 32; ++t) {
              const float x0 = keys(w0) ? __uint_as_float(o[t]) * w0 : 0.f;
              o[t] = __float_as_uint(keys(w1) ? fmaf(__uint_as_float(o1[t]), w1, x0) : x0);
            }
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 32; ++t) o[t] = __float_as_uint(keys(w0) ? __uint_as_float(o[t]) * w0 : 0.f);
          }
          if (valid) {
            if (part >= 0) {
              float4* op = reinterpret_cast<float4*>(a.part_o + prow * DV) + c * 8;
#pragma unroll
              for (int t = 0; t < 8; ++t)
                op[t] = make_float4(__uint_as_float(o[4 * t]), __uint_as_float(o[4 * t + 1]), __uint_as_float(o[4 * t + 2]),
                                    __uint_as_float(o[4 * t + 3]));
            } else {
              uint32_t pw[16];
#pragma unroll
              for (int t = 0; t < 16; ++t) pw[t] = pack_bf16x2(__uint_as_float(o[2 * t]), __uint_as_float(o[2 * t + 1]));
              store_row64(orow + c * 32, pw);
            }
          }
        }
        if (valid && (!dual || i == 0)) {
          if (part >= 0) a.part_lse[prow] = lse2;
          else a.lse[static_cast<int64_t>(head) * a.total_q + w.q_row + tok] = lse2 * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar->o_free);
        mbar_arrive(&bar->seg_empty[seg_i % kSegs]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

// Merges the units that were cut, launched while paged_kernel still runs (it waits for
// it below): with the segments' LSE_r in log2 units, M their
// maximum, O = sum_r 2^(LSE_r - M) O_r / sum_r 2^(LSE_r - M), the segments in key
// order within a warp and then warp after warp. Bound by latency (a segment's O is loaded beside its LSE: one request
// of 4100 tokens 13.9 us, 14.6 with the loads one after the other): WPR warps share a row,
// each taking every WPR-th segment (8 where rows are few, as in decoding, else 1); lane l
// holds columns [DV/32 l, DV/32 (l + 1)).
template <int DV, int WPR>
__global__ void __launch_bounds__(256) merge_kernel(const PagedArgs a) {
  constexpr int CPL = DV / 32;
  __shared__ float s_acc[WPR > 1 ? WPR : 1][DV];
  __shared__ float s_sum[WPR > 1 ? WPR : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MergeUnit m = a.merge[blockIdx.x];
  if (m.n < 1) return;
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int rr = WPR > 1 ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y * 8 + warp);
  const int part = WPR > 1 ? warp : 0;
  if (rr >= m.ntok * a.kv_group) return;  // (whole blocks where WPR > 1)
  const int tok = rr / a.kv_group, hd = rr - tok * a.kv_group, tile = tok / a.tile_tokens;
  const int row = tile * BM + (tok - tile * a.tile_tokens) * a.kv_group + hd;
  auto at = [&](int r) -> int64_t {
    return static_cast<int64_t>(r == 0 ? m.first : m.rest + r - 1) * a.part_rows + row;
  };
  // the first segments' O, loaded beside their LSE
  using Vec = std::conditional_t<CPL == 4, float4, float2>;
  auto load_o = [&](int r) -> Vec { return *reinterpret_cast<const Vec*>(a.part_o + at(r) * DV + lane * CPL); };
  constexpr int kAhead = 4;
  Vec ahead[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (part + u * WPR < m.n) ahead[u] = load_o(part + u * WPR);
  const float lse0 = lane < m.n ? a.part_lse[at(lane)] : -INFINITY;  // segment `lane`'s
  float mx = lse0;
  // (a segment's NaN is kept: dropped, the row would pass for one without keys, or for the other segments' alone)
  for (int r = lane + 32; r < m.n; r += 32) mx = fmax_nan(mx, a.part_lse[at(r)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  float sum = 0.f, acc[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) acc[c] = 0.f;
  if (mx != -INFINITY) {
    auto add = [&](int r, const Vec& v) {
      const float wr = ex2_mufu((r < 32 ? __shfl_sync(0xffffffffu, lse0, r & 31) : a.part_lse[at(r)]) - mx);
      sum += wr;
      acc[0] = fmaf(wr, v.x, acc[0]);
      acc[1] = fmaf(wr, v.y, acc[1]);
      if constexpr (CPL == 4) {
        acc[2] = fmaf(wr, v.z, acc[2]);
        acc[3] = fmaf(wr, v.w, acc[3]);
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (part + u * WPR < m.n) add(part + u * WPR, ahead[u]);
#pragma unroll 4
    for (int r = part + kAhead * WPR; r < m.n; r += WPR) add(r, load_o(r));
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) s_acc[warp][lane * CPL + c] = acc[c];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      sum += s_sum[w];
#pragma unroll
      for (int c = 0; c < CPL; ++c) acc[c] += s_acc[w][lane * CPL + c];
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int64_t head = static_cast<int64_t>(m.hk) * a.kv_group + hd;
  __nv_bfloat16* o = a.o + static_cast<int64_t>(m.q_row + tok) * a.o_row + head * a.o_head + lane * CPL;
  if constexpr (CPL == 4)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) a.lse[head * a.total_q + m.q_row + tok] = sum != 0.f ? (mx + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// The list of paged_kernel<EVEN = false>: first the parts of the units (request, 2 *
// tile_tokens tokens, K/V head) that cost more than an equal share of the whole (cost:
// key blocks, doubled for two tiles of rows), cut evenly; then one entry per unit (that
// of a cut unit is empty), requests with the most keys first (a counting sort by key
// blocks), a request's last tokens, which see the most keys, before its first, the K/V
// heads of the same tokens side by side. One block; the order affects only scheduling.
// Bound by latency: requests with few units are written by one thread each, the others
// by a warp.
constexpr int kListThreads = 1024, kBins = 2048;

__global__ void __launch_bounds__(kListThreads, 1) chunk_list_kernel(const PagedArgs a, int ctas) {
  __shared__ int bins[kBins];
  __shared__ long long sums[kListThreads / 32];
  __shared__ int warp_items[kListThreads / 32];
  __shared__ int large[kListThreads];  // requests for the warps: (request, first entry)
  __shared__ int large_at[kListThreads];
  __shared__ int n_slots, n_merge, n_parts, n_large;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // paged_kernel sets itself up meanwhile
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int unit_tokens = 2 * a.tile_tokens;
  for (int x = tid; x < kBins; x += kListThreads) bins[x] = 0;
  if (tid == 0) n_slots = n_merge = n_parts = n_large = 0;
  __syncthreads();
  auto bin_of = [&](const Bounds& b) { return kBins - 1 - min(kBins - 1, ceil_div(b.nk, BN)); };  // most keys first
  // The whole's cost, bounded from above in closed form: over a request's u units the keys seen by
  // a unit's last token sum to at most u nk, and causally, where unit u - 1 - m ends more than
  // (m - 1) unit_tokens before the request does, to at most u nk - unit_tokens (u - 1) (u - 2) / 2.
  long long w = 0;
  for (int s = tid; s < a.num_seqs; s += kListThreads) {
    const Bounds b = bounds(a, s);
    if (b.nq == 0) continue;
    const long long u = (b.nq + unit_tokens - 1) / unit_tokens;
    long long keys = u * b.nk;
    if (a.causal && b.nk >= b.nq) keys -= unit_tokens * ((u - 1) * (u - 2) / 2);
    w += 2 * ((keys >> 7) + u + 1);
    atomicAdd(&bins[bin_of(b)], static_cast<int>(u) * a.heads_kv);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
  if (lane == 0) sums[warp] = w;
  __syncthreads();
  w = 0;
#pragma unroll
  for (int x = 0; x < kListThreads / 32; ++x) w += sums[x];
  w *= a.heads_kv;
  // an equal share of the work (a unit costs less than 2^26)
  const uint32_t cap = static_cast<uint32_t>(
      min(max(static_cast<long long>(kPagedMinItem), (w + ctas - 1) / ctas), static_cast<long long>(1) << 30));
  // bins -> first entry of each bin: two bins per thread, a scan per warp and over the warps' sums
  const int b0 = bins[2 * tid], b1 = bins[2 * tid + 1];
  int inc = b0 + b1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) warp_items[warp] = inc;
  __syncthreads();
  int before = inc - b0 - b1, total = 0;
#pragma unroll
  for (int x = 0; x < kListThreads / 32; ++x) {
    const int y = warp_items[x];
    if (x < warp) before += y;
    total += y;
  }
  bins[2 * tid] = before;
  bins[2 * tid + 1] = before + b0;
  __syncthreads();
  const int first_unit = 2 * ctas;  // the cut units' parts come before
  // entry x (of units * heads_kv) of request s, whose entries begin at `at`
  auto write = [&](int s, const Bounds& b, int units, int at, int x) {
    const int u = units - 1 - x / a.heads_kv, hk = x % a.heads_kv;  // the last tokens first
    const int tok0 = u * unit_tokens, ntok = min(unit_tokens, b.nq - tok0);
    const int nb = unit_blocks(a, b, tok0 + ntok - 1);
    const uint32_t cost = static_cast<uint32_t>(nb) * (ntok > a.tile_tokens ? 2u : 1u);
    ChunkItem it{s, hk, tok0, 0, nb, -1};
    if (cost > cap) {
      // fewer than `ctas` units cost more than a share (the costs sum to at most ctas shares), and
      // their cuts number at most cost / share + 1 each: below 2 * ctas in all
      const int k = static_cast<int>((cost + cap - 1) / cap);
      const int slot = atomicAdd(&n_slots, k), at_part = atomicAdd(&n_parts, k);
      a.merge[atomicAdd(&n_merge, 1)] = MergeUnit{b.q0 + tok0, ntok, hk, slot, slot + 1, k};
      for (int y = 0; y < k; ++y)
        a.items[at_part + y] = ChunkItem{s, hk, tok0, static_cast<int>(static_cast<long long>(nb) * y / k),
                                         static_cast<int>(static_cast<long long>(nb) * (y + 1) / k), slot + y};
      it.seq = -1;
    }
    const int i = first_unit + at + x;
    if (i < a.items_bound) a.items[i] = it;
  };
  for (int s = tid; s < a.num_seqs; s += kListThreads) {
    const Bounds b = bounds(a, s);
    if (b.nq == 0) continue;
    const int units = ceil_div(b.nq, unit_tokens), n = units * a.heads_kv;
    const int at = atomicAdd(&bins[bin_of(b)], n);
    if (n > 16) {
      const int x = atomicAdd(&n_large, 1);
      if (x < kListThreads) {
        large[x] = s;
        large_at[x] = at;
        continue;
      }
    }
    for (int x = 0; x < n; ++x) write(s, b, units, at, x);
  }
  __syncthreads();
  for (int y = warp; y < min(n_large, kListThreads); y += kListThreads / 32) {
    const Bounds b = bounds(a, large[y]);
    const int units = ceil_div(b.nq, unit_tokens);
    for (int x = lane; x < units * a.heads_kv; x += 32) write(large[y], b, units, large_at[y], x);
  }
  __syncthreads();
  for (int x = tid; x < ctas; x += kListThreads)
    if (x >= n_merge) a.merge[x].n = 0;
  if (tid == 0) {
    a.list->n_parts = n_parts;
    a.list->n_items = n_parts + min(total, a.items_bound - first_unit);
    a.list->next = ctas;
  }
}

template <int DQK, int DV, int MOD, bool EVEN>
cudaError_t launch_main(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                        cudaStream_t stream) {
  using C = Cfg<DQK, DV, EVEN>;
  auto kern = paged_kernel<DQK, DV, MOD, EVEN>;
  static PerDeviceOnce once;
  const cudaError_t e = once.run([&]() -> cudaError_t {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (r != cudaSuccess) return r;
    cudaFuncAttributes fa{};
    r = cudaFuncGetAttributes(&fa, kern);
    if (r != cudaSuccess) return r;
    // The setmaxnreg split must fit in the registers the CTA is launched with.
    return fa.numRegs * kThreads < C::REG_BUDGET ? cudaErrorInvalidConfiguration : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  if constexpr (EVEN) {
    kern<<<ctas, kThreads, C::SMEM, stream>>>(tq, tk, tv, a);
    return cudaGetLastError();
  }
  return launch_early(kern, dim3(ctas), kThreads, C::SMEM, stream, tq, tk, tv, a);  // behind chunk_list_kernel
}

template <int DQK, int DV>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, bool even,
                     bool decode, int ctas, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (!even) {
    chunk_list_kernel<<<1, kListThreads, 0, stream>>>(a, ctas);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (decode) {
    e = launch_paged_decode(DQK, DV, tq, tk, tv, a, ctas, stream);
  } else switch (a.score_mod) {
    case kModNone:
      e = even ? launch_main<DQK, DV, kModNone, true>(tq, tk, tv, a, ctas, stream)
               : launch_main<DQK, DV, kModNone, false>(tq, tk, tv, a, ctas, stream);
      break;
    case kModSoftcap:
      e = even ? launch_main<DQK, DV, kModSoftcap, true>(tq, tk, tv, a, ctas, stream)
               : launch_main<DQK, DV, kModSoftcap, false>(tq, tk, tv, a, ctas, stream);
      break;
    case kModAlibi:
      e = even ? launch_main<DQK, DV, kModAlibi, true>(tq, tk, tv, a, ctas, stream)
               : launch_main<DQK, DV, kModAlibi, false>(tq, tk, tv, a, ctas, stream);
      break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  const int rows = min(a.max_q, (even ? 1 : 2) * a.tile_tokens) * a.kv_group;
  // Up to 16 rows, whose blocks fit the GPU at once, eight warps share a row: 16 rows over 16000 keys 13.0 us, with one warp
  // 22.8, over 1000 11.4 and 10.2. (32 rows: over 16000 16.3 and 25.2, over 1000 13.4 and 10.8; 33 requests of 3 to 6 tokens
  // 36.9 and 29.5. The segments decide, which the host does not know.)
  if (rows <= 16)
    return launch_early(merge_kernel<DV, 8>, dim3(ctas, rows), 256, 0, stream, a);
  return launch_early(merge_kernel<DV, 1>, dim3(ctas, (rows + 7) / 8), 256, 0, stream, a);
}

}  // namespace paged

cudaError_t launch_fwd_paged(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedArgs& a, bool even, bool decode, int ctas, cudaStream_t stream) {
  if (ctas < 1 || a.merge == nullptr || a.part_o == nullptr || (!even && a.items == nullptr)) return cudaErrorInvalidValue;
  if (d_qk == 64 && d_v == 64) return paged::launch_d<64, 64>(tq, tk, tv, a, even, decode, ctas, stream);
  if (d_qk == 128 && d_v == 128) return paged::launch_d<128, 128>(tq, tk, tv, a, even, decode, ctas, stream);
  if (d_qk == 192 && d_v == 128) return paged::launch_d<192, 128>(tq, tk, tv, a, even, decode, ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
