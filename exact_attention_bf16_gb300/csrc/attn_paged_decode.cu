// attn_fwd_paged for few rows per K/V head (decoding): up to N = 16 rows (token, head of
// the group) per request.
//
// The products are taken the other way round than in attn_paged.cu, with the long
// side in the 128 lanes of an MMA:
//   S^T [128 keys x N rows]  = K Q^T       (A = K block, B = Q, both K-major)
//   O^T [d_v x N rows]      += V^T P^T     (A = V block read M-major, B = P, K-major)
// so that a tile's softmax is spread over 128 threads, one key each with N values,
// instead of N threads with 128, and an MMA is N wide instead of 128. The running
// maximum of a row is then a maximum across threads; it is needed only when some
// logit exceeds the one in use by more than 8 (log2 units), so per block the four
// warps only vote on that (one named barrier), and the maxima, the rescale of O^T
// and of the sums run when the vote says so (a row's first block, rarely later). Row
// sums stay per thread (per key lane) until the end.
//
// Bound by HBM: per 128 keys and K/V head at d = 128 64 KB against 16 MMAs of about
// 50 cycles. 64 requests of up to 32768 tokens, 32 heads over 8, d = 128: 307 us, 6.67 TB/s
// (98% of a copy's), 321 us by paged_kernel; one of 4100 tokens 13.9 us against 15, its
// launches, first copies and merge. d = 64 (8 heads of their own, 64 requests) reaches 4.2 TB/s
// against 3.8: a 128-key block is half the bytes for the same waits. (192, 128): 6.3 TB/s.
// With 32 columns the same calls took 341 us where 16 took 323 and paged_kernel 332 (64
// requests, 8 heads, d = 128), with 64 columns 416, so 17 rows and more are paged_kernel's. Up
// to 16 rows of the other head sizes, here and there: d = 64, 8 requests of 8000 tokens 33.4 us
// and 37.7, one of 4100 13.7 both (16 rows 15.2 and 15.0); (192, 128), one 14.1 and 15.4, 64
// requests 479 and 484. Work is the even split of paged_common.cuh; two streams over the even
// and the odd key blocks hide the chain S^T -> softmax -> O^T, as there.
//
// A relative position bias is 16 loads a key lane and block, ahead of the block's logits: 64 requests of 300 to 16384 tokens, 32
// heads over 8, d = 128: 206 us, 200 without a bias, 256 by paged_kernel with one.
//
// Warps: 0 work and TMA copies, 1 MMA issue, 4..7 and 8..11 softmax of stream 0 and 1.
#include <cstddef>

#include "kernels.h"
#include "paged_common.cuh"
#include "ptx_sm100.cuh"
#include "rel_bias.cuh"
#include "score_mod.cuh"

namespace gb300 {
namespace paged {
namespace decode {

constexpr int N = kDecodeRows;

template <int DQK, int DV>
struct Cfg {
  static constexpr int QCH = DQK / 64, VCH = DV / 64;
  static constexpr int K_BYTES = QCH * kChunk, V_BYTES = VCH * kChunk;
  static constexpr int Q_CHUNK = N * 128, Q_BYTES = QCH * Q_CHUNK;  // 64 columns of N rows
  static constexpr int P_CHUNK = N * 128, P_BYTES = 2 * P_CHUNK;    // 64 keys of N rows; [N][128 keys]
  static constexpr int NQ = 2;  // the next segment's Q is copied while this one's is used
  // ring slots: what 227 KB hold beside Q and P
  static constexpr int NK = DQK == 64 ? 6 : (DQK == 128 ? 3 : 2);
  static constexpr int NV = DQK == 64 ? 6 : 3;
  static constexpr int OFF_V = NK * K_BYTES;
  static constexpr int OFF_Q = OFF_V + NV * V_BYTES;
  static constexpr int OFF_P = OFF_Q + NQ * Q_BYTES;
  static constexpr int OFF_M = OFF_P + 2 * P_BYTES;  // [2 streams][N]: the maxima in use (log2 units)
  static constexpr int OFF_W = OFF_M + 2 * N * 4;    // [2 streams][4 warps][N]: warps' maxima, rescales, then sums
  static constexpr int OFF_SEG = OFF_W + 2 * 4 * N * 4;
  static constexpr int OFF_BAR = OFF_SEG + kSegs * 64;
  static constexpr int SMEM = OFF_BAR + 640;  // the base is 1024-byte aligned (checked)
  static_assert(SMEM <= 232448, "shared memory budget");
  // TMEM columns: S^T and O^T of the two streams
  static constexpr uint32_t tS(int i) { return N * i; }
  static constexpr uint32_t tO(int i) { return 2 * N + N * i; }
  static constexpr uint32_t COLS = 4 * N;  // a power of two
  static constexpr int M_O = DV;           // rows of O^T (DV = 64: an M = 64 MMA)
};

struct Bars {
  // one arrival
  uint64_t q_full[2], q_free[2];
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], o_full[2];
  uint64_t seg_full[kSegs];
  uint64_t mma_done;
  // four: a warpgroup's warps
  uint64_t p_full[2];
  uint64_t x_full[2];  // a stream's maxima and sums are in shared memory
  // nine: eight softmax warps and the MMA thread
  uint64_t seg_empty[kSegs];
  uint64_t o_free;     // a segment is over: its O has been read, its MMAs issued (so neither side gets two ahead)
  uint32_t tmem_base;
  EvenStart even;
};
static_assert(sizeof(Bars) <= 640, "barriers must fit their reserved bytes");

// Named barrier of one warpgroup with the OR of its threads' predicates. Every wait that
// precedes one is bounded and its failure goes into a vote, so all warps get here.
__device__ __forceinline__ bool group_any(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(id) : "memory");
}

// Reduces 16 values per lane over the warp and writes the results to out[0 .. 16). At each step
// a lane keeps one half of its columns and hands over the other: 16 shuffles, not 80.
template <typename Op>
__device__ __forceinline__ void warp_reduce_cols(const float (&x)[N], uint32_t lane, float* out, Op op) {
  static_assert(N == 16, "lanes 2c and 2c + 1 end with the halves of column c");
  float v[N];
#pragma unroll
  for (int c = 0; c < N; ++c) v[c] = x[c];
#pragma unroll
  for (int st = 0; (N >> (st + 1)) > 0; ++st) {
    const int half = N >> (st + 1);
    const uint32_t bit = 16u >> st;
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
      if (c < half) {
        const float send = up ? v[c] : v[c + half], keep = up ? v[c + half] : v[c];
        v[c] = op(keep, __shfl_xor_sync(0xffffffffu, send, bit));
      }
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
  if ((lane & 1u) == 0) out[lane >> 1] = v[0];
}

// MOD: kModNone or kModRelBias.
template <int DQK, int DV, int MOD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv, const PagedArgs a) {
  using C = Cfg<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {  // the 128-byte-swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(a.status, DEV_BAD_CONFIG, 0x4000);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sQ = smem + C::OFF_Q;
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
    tmem_alloc(&bar->tmem_base, C::COLS);
    tmem_relinquish();
  }
  // rows of Q that no copy writes: zeros, whose logits never move a maximum
  for (int x = static_cast<int>(threadIdx.x); x < C::NQ * C::Q_BYTES / 16; x += kThreads)
    reinterpret_cast<uint4*>(sQ)[x] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  even_split(a, &bar->even);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bar->tmem_base;
  if constexpr (MOD == kModRelBias) asm volatile("griddepcontrol.wait;" ::: "memory");  // the bias's layout
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // merge_kernel, as SMs become free

  if (warp == 0) {
    // ===================== work and copies ==================================
    const uint32_t q_bytes = static_cast<uint32_t>(a.kv_group * a.q_box_tokens) * 128u * C::QCH;
    Ring<C::NQ> rq;
    uint32_t cq = 0;
    EvenWalk walk;
    walk.begin(a, &bar->even);
    const bool ok = copy_loop<C>(
        a, bar, sSeg, sK, sV, &tmk, &tmv, 0x4100, [&] { return walk.next(a, &bar->even); },
        [&](const Seg& w) {
          if (!mbar_wait_warp(&bar->q_free[rq.slot], rq.phase ^ 1u, a.status, 0x4120)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&bar->q_full[rq.slot], q_bytes);
          __syncwarp();
          if (static_cast<int>(lane) < C::QCH)
            tma_load_4d(sQ + rq.slot * C::Q_BYTES + lane * C::Q_CHUNK, &tmq, &bar->q_full[rq.slot],
                        static_cast<int>(lane) * 64, w.hk * a.kv_group, w.q_row, 0);
          rq.next();
          ++cq;
          return true;
        });
    walk.finish(a);
    if (!ok)
      for (uint32_t u = 0; u < C::NQ && u < cq; ++u)
        mbar_wait(&bar->q_full[(cq - 1 - u) % C::NQ], ((cq - 1 - u) / C::NQ) & 1u, nullptr, 0);
  } else if (warp == 1) {
    if (lane == 0) {
      // ===================== MMA issue ======================================
      constexpr uint32_t idS = idesc_bf16_f32(BN, N, false, false);
      constexpr uint32_t idO = idesc_bf16_f32(C::M_O, N, true, false);
      Ring<C::NK> rk;
      Ring<C::NV> rv;
      Ring<C::NQ> rq;
      uint32_t seg_i = 0, pp = 0;  // pp: a bit per stream
      bool ok = true;
      const uint64_t dk0 = smem_desc(smem_u32(sK), 16, 1024, SWZ_128B), dq0 = smem_desc(smem_u32(sQ), 16, 1024, SWZ_128B);
      const uint64_t dv0 = smem_desc(smem_u32(sV), kChunk, 1024, SWZ_128B);
      const uint64_t dp0 = smem_desc(smem_u32(smem + C::OFF_P), 16, 1024, SWZ_128B);
      for (;;) {
        const int slot = static_cast<int>(seg_i % kSegs);
        ok = mbar_wait(&bar->seg_full[slot], (seg_i / kSegs) & 1u, a.status, 0x4200);
        if (!ok) break;
        const int more = sSeg[slot].more, n = sSeg[slot].n0;
        mbar_arrive(&bar->seg_empty[slot]);
        if (!more) break;
        // the previous segment's O has been read: before the first PV overwrites it
        auto wait_o = [&]() { return seg_i == 0 || mbar_wait(&bar->o_free, (seg_i - 1) & 1u, a.status, 0x4210); };
        if (n == 0) ok = wait_o();
        const uint64_t dq = desc_add(dq0, rq.slot * C::Q_BYTES);
        for (int j = 0; j <= n && n > 0 && ok; ++j) {
          if (j < n) {
            ok = mbar_wait(&bar->k_full[rk.slot], rk.phase, a.status, 0x4220);
            if (ok && j == 0) ok = mbar_wait(&bar->q_full[rq.slot], rq.phase, a.status, 0x4230);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dk = desc_add(dk0, rk.slot * C::K_BYTES);
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk)
              mma_ss(tbase + C::tS(j & 1), desc_add(dk, (kk / 4) * kChunk + (kk % 4) * 32),
                     desc_add(dq, (kk / 4) * C::Q_CHUNK + (kk % 4) * 32), idS, kk > 0 ? 1u : 0u);
            mma_commit(&bar->s_full[j & 1]);  // (also says that K(j) and V(j - 2) have been read)
            if (j == n - 1) mma_commit(&bar->q_free[rq.slot]);
            rk.next();
          }
          if (j > 0) {
            const int i = (j - 1) & 1;
            if (j == 1) ok = wait_o();
            ok = ok && mbar_wait(&bar->v_full[rv.slot], rv.phase, a.status, 0x4240) &&
                 mbar_wait(&bar->p_full[i], (pp >> i) & 1u, a.status, 0x4250);
            if (!ok) break;
            tc_fence_after();
            pp ^= 1u << i;
            const uint64_t dv = desc_add(dv0, rv.slot * C::V_BYTES), dp = desc_add(dp0, i * C::P_BYTES);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)  // 16 keys: 16 rows of V, 32 bytes of P's rows
              mma_ss(tbase + C::tO(i), desc_add(dv, kk * 2048),
                     desc_add(dp, (kk / 4) * C::P_CHUNK + (kk % 4) * 32), idO, (kk > 0 || j > 2) ? 1u : 0u);
            if (j - 1 >= n - 2) mma_commit(&bar->o_full[i]);
            rv.next();
          }
        }
        if (!ok) break;
        mbar_arrive(&bar->o_free);
        if (n > 0) rq.next();
        ++seg_i;
      }
      mma_commit(&bar->mma_done);
      mbar_wait(&bar->mma_done, 0, a.status, 0x42ff);
    }
  } else if (warp >= 4) {
    // ======================= softmax and output =============================
    const int i = (static_cast<int>(warp) - 4) / 4;  // stream
    const uint32_t quarter = warp & 3u;
    const int key_lane = static_cast<int>(quarter * 32 + lane);  // this thread's key of a block
    const uint32_t lane_base = tbase + ((quarter * 32u) << 16);
    const int bid = 1 + i;  // named barrier of this warpgroup
    float* sM = reinterpret_cast<float*>(smem + C::OFF_M) + i * N;
    float* sW = reinterpret_cast<float*>(smem + C::OFF_W) + i * 4 * N;
    // P [N rows][128 keys]: this thread's column; 16-byte pieces swizzled by the row
    uint8_t* sP = smem + C::OFF_P + i * C::P_BYTES + (key_lane / 64) * C::P_CHUNK + (key_lane % 8) * 2;
    const int piece = (key_lane % 64) / 8;
    const float sl2 = a.scale_log2;
    bool ok = true;
    for (uint32_t seg_i = 0;; ++seg_i) {
      // (a copy: read by all lanes before the warp lets the slot go, below)
      const volatile Seg& w = sSeg[seg_i % kSegs];
      ok = ok && mbar_wait_warp(&bar->seg_full[seg_i % kSegs], (seg_i / kSegs) & 1u, a.status, 0x4300);
      // every warp has left the segment before: its reads of sM and sW of both streams are done
      if (ok && seg_i > 0) ok = mbar_wait_warp(&bar->o_free, (seg_i - 1) & 1u, a.status, 0x4328);
      if (group_any(bid, !ok) || !w.more) break;  // (a wait that failed anywhere in the segment before, too)
      const int n = w.n0, nk = w.nk, pos0 = w.pos0, kt0 = w.kt0;
      const int full = a.causal ? min(nk, max(0, pos0 + 1)) : nk;  // keys that every row sees
      auto page_ok = [&](int key) -> bool {
        if (key >= nk) return true;
        const int pg = __ldg(a.block_table + w.seq * a.block_table_stride + (key >> a.page_shift));
        return pg >= 0 && pg < a.num_pages;
      };
      float l[N];  // this key lane's share of the row sums
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.f;
      uint32_t s_phase = i == 0 ? w.s0 : w.s1;
      bool pg_ok = i < n ? page_ok((kt0 + i) * BN + key_lane) : true;
      for (int j = i; j < n; j += 2, ++s_phase) {
        const int key = (kt0 + j) * BN + key_lane;
        const bool here = pg_ok;
        if (j + 2 < n) pg_ok = page_ok(key + 2 * BN);  // fetched one block ahead
        // relative position bias of this key to each column's query (a load per column, the same for all lanes beyond the reach)
        float bias[N];
        if constexpr (MOD == kModRelBias) {
          const int width = 2 * a.rel.reach + 2 * kRelPad;
          const float* row = a.rel.by_place + static_cast<int64_t>(w.hk) * a.kv_group * width + a.rel.reach + kRelPad;
          int r = key - pos0, hd = 0;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            bias[c] = __ldg(row + static_cast<int64_t>(hd) * width + max(-a.rel.reach, min(a.rel.reach, r)));
            if (++hd == a.kv_group) hd = 0, --r;
          }
        }
        ok = ok && mbar_wait_warp(&bar->s_full[i], s_phase & 1u, a.status, 0x4310 + i);
        // a commit costs the MMA thread several hundred cycles, so the slots are released from here: S(j) of
        // block j follows PV(j - 2) in issue order, so K(j) and V(j - 2) have been read
        if (ok && quarter == 0 && lane == 0) {
          mbar_arrive(&bar->k_empty[(w.v0 + j) % C::NK]);
          if (j >= 2) mbar_arrive(&bar->v_empty[(w.v0 + j - 2) % C::NV]);
        }
        tc_fence_after();
        uint32_t sr[N];
        tmem_ld16(lane_base + C::tS(i), sr);
        tmem_wait_ld();
        float s[N];
#pragma unroll
        for (int c = 0; c < N; ++c)
          s[c] = (MOD == kModRelBias ? __uint_as_float(sr[c]) + bias[c] : __uint_as_float(sr[c])) * sl2;
        if (!here || key >= full) {  // keys that no row or not every row sees
          int tok = 0, left = a.kv_group;  // of column c
#pragma unroll
          for (int c = 0; c < N; ++c) {
            if (!here || key >= nk || (a.causal && key > pos0 + tok)) s[c] = -INFINITY;
            if (--left == 0) left = a.kv_group, ++tok;
          }
        }
        // does any logit exceed the maximum in use by more than the threshold?
        const bool fresh = j == i;
        bool over = fresh || !ok;
        if (!fresh) {
          float t = -INFINITY;
#pragma unroll
          for (int c = 0; c < N; c += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(sM + c);
            t = fmax3(t, s[c] - m4.x, s[c + 1] - m4.y);
            t = fmax3(t, s[c + 2] - m4.z, s[c + 3] - m4.w);
          }
          over = over || t > kThreshold;
        }
        if (group_any(bid, over)) {
          if (group_any(bid, !ok)) {  // a wait ran out in some warp: leave together
            ok = false;
            break;
          }
          warp_reduce_cols(s, lane, sW + quarter * N, [](float x, float y) { return fmaxf(x, y); });
          group_sync(bid);
          if (key_lane < N) {  // one thread per row: the maximum in use is replaced where the block exceeds it enough
            const int c = key_lane;
            const float m_blk = fmaxf(fmaxf(sW[c], sW[N + c]), fmaxf(sW[2 * N + c], sW[3 * N + c]));
            const float m_old = fresh ? -INFINITY : sM[c];
            const bool need = m_blk > m_old + kThreshold;
            sW[c] = !need ? 1.f : (m_old == -INFINITY ? 0.f : ex2_mufu(m_old - m_blk));
            sM[c] = need ? m_blk : m_old;
          }
          group_sync(bid);
          if (!fresh) {
            uint32_t o[N];
            tmem_ld16(lane_base + C::tO(i), o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < N; ++c) {
              const float alpha = sW[c];
              l[c] *= alpha;
              o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            }
            tmem_st16(lane_base + C::tO(i), o);
            tmem_wait_st();
          }
          group_sync(bid);
        }
        // P = 2^(s - m), a column of P per thread; a row without keys so far has m = -inf: p = 0
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(sM + c);
          const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float p = ex2_mufu(s[c + u] - (mm[u] == -INFINITY ? 0.f : mm[u]));
            l[c + u] += p;
            *reinterpret_cast<__nv_bfloat16*>(sP + (c + u) * 128 + ((piece ^ ((c + u) & 7)) << 4)) = __float2bfloat16_rn(p);
          }
        }
        // The request's last block: cache rows past its last key, on the page that holds it, may be
        // anything (0 x NaN is NaN), so they are zeroed before the PV product reads them.
        const int tail = nk - (kt0 + j) * BN;  // keys of the request in this block
        if (tail < BN && tail > 0 && (tail & (a.page_size - 1)) != 0) {
          const uint32_t u = w.v0 + static_cast<uint32_t>(j), vs = u % C::NV;
          ok = ok && mbar_wait_warp(&bar->v_full[vs], (u / C::NV) & 1u, a.status, 0x4320);
          const int end = min(BN, (tail | (a.page_size - 1)) + 1);
          uint8_t* v = sV + vs * C::V_BYTES;
          const int units = (end - tail) * 8;  // 16-byte pieces of a chunk
          for (int x = key_lane; x < units * C::VCH && ok; x += 128)
            *reinterpret_cast<uint4*>(v + (x / units) * kChunk + tail * 128 + (x % units) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[i]);
      }
      // ---- output: sums over the key lanes, the two streams merged
      if (ok) {
        warp_reduce_cols(l, lane, sW + quarter * N, [](float x, float y) { return x + y; });
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->x_full[i]);
        const uint32_t xp = (w.phase >> 2) & 1u;
        ok = mbar_wait_warp(&bar->x_full[i], xp, a.status, 0x4330) &&
             mbar_wait_warp(&bar->x_full[1 - i], xp, a.status, 0x4331);
      }
      // (the exchange also says that the other warpgroup has left the segment before, so that
      // its O barrier is at most one phase behind)
      if (ok && n > 0) ok = mbar_wait_warp(&bar->o_full[0], w.phase & 1u, a.status, 0x4340);
      if (ok && n > 1) ok = mbar_wait_warp(&bar->o_full[1], (w.phase >> 1) & 1u, a.status, 0x4341);
      if (ok) {
        tc_fence_after();
        if (i == 0 && quarter == 0 && lane == 0) {  // the last two V blocks
          if (n > 1) mbar_arrive(&bar->v_empty[(w.v0 + n - 2) % C::NV]);
          if (n > 0) mbar_arrive(&bar->v_empty[(w.v0 + n - 1) % C::NV]);
        }
        // this warpgroup writes rows [i N/2, (i + 1) N/2); lane u of each warp holds row i N/2 + u's weights
        const float* m_of = reinterpret_cast<const float*>(smem + C::OFF_M);
        const float* l_of = reinterpret_cast<const float*>(smem + C::OFF_W);
        constexpr int HALF = N / 2;
        const int row = i * HALF + static_cast<int>(lane) % HALF;
        const int rows = w.ntok * a.kv_group, part = w.part;
        float la = 0.f, lb = 0.f, ma = -INFINITY, mb = -INFINITY;
        if (n > 0) {
          ma = m_of[row];
          la = (l_of[row] + l_of[N + row]) + (l_of[2 * N + row] + l_of[3 * N + row]);
        }
        if (n > 1) {
          mb = m_of[N + row];
          lb = (l_of[4 * N + row] + l_of[5 * N + row]) + (l_of[6 * N + row] + l_of[7 * N + row]);
        }
        const float mm = fmaxf(ma, mb);
        // (a sum of 0 is a row without keys; a NaN sum is no such row, and stays NaN in O and LSE)
        const float ea = la != 0.f ? ex2_mufu(ma - mm) : 0.f, eb = lb != 0.f ? ex2_mufu(mb - mm) : 0.f;
        const float lt = la * ea + lb * eb;
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        const float w0 = ea * inv, w1 = eb * inv;
        const float lse2 = lt != 0.f ? mm + log2f(lt) : -INFINITY;
        // A stream in which the row saw no key (or that has no block) adds nothing, also where its values are not finite
        // (0 x NaN).
        const uint32_t keys0 = __ballot_sync(0xffffffffu, la != 0.f), keys1 = __ballot_sync(0xffffffffu, lb != 0.f);
        const int q_row = w.q_row, head0 = w.hk * a.kv_group;
        if (quarter == 0 && static_cast<int>(lane) < HALF && row < rows) {
          const int tok = row / a.kv_group;
          if (part >= 0)
            a.part_lse[static_cast<int64_t>(part) * a.part_rows + row] = lse2;
          else
            a.lse[static_cast<int64_t>(head0 + row - tok * a.kv_group) * a.total_q + q_row + tok] =
                lse2 * 0.69314718055994531f;
        }
        // O^T: lane = column of O (d_v = 64: an M = 64 product, whose row m is in lane 32 (m / 16) + m % 16)
        const bool has_col = DV == 128 || lane < 16;
        const int col = DV == 128 ? key_lane : static_cast<int>(quarter * 16 + lane);
        if (i * HALF < rows) {
          uint32_t o0[HALF], o1[HALF];
          tmem_ld8(lane_base + C::tO(0) + i * HALF, o0);  // (columns never written are not used)
          tmem_ld8(lane_base + C::tO(1) + i * HALF, o1);
          tmem_wait_ld();
          int tok = i * HALF / a.kv_group, hd = i * HALF - tok * a.kv_group;
#pragma unroll
          for (int c = 0; c < HALF; ++c) {
            const float x0 = __shfl_sync(0xffffffffu, w0, c), x1 = __shfl_sync(0xffffffffu, w1, c);
            const float v0 = (keys0 >> c) & 1u ? __uint_as_float(o0[c]) * x0 : 0.f;
            const float v = (keys1 >> c) & 1u ? fmaf(__uint_as_float(o1[c]), x1, v0) : v0;
            const int rw = i * HALF + c;
            if (rw < rows && has_col) {
              if (part >= 0)
                a.part_o[(static_cast<int64_t>(part) * a.part_rows + rw) * DV + col] = v;
              else
                a.o[static_cast<int64_t>(q_row + tok) * a.o_row + static_cast<int64_t>(head0 + hd) * a.o_head + col] =
                    __float2bfloat16_rn(v);
            }
            if (++hd == a.kv_group) hd = 0, ++tok;
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0 && ok) {
        mbar_arrive(&bar->o_free);
        mbar_arrive(&bar->seg_empty[seg_i % kSegs]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, C::COLS);
}

template <int DQK, int DV, int MOD>
cudaError_t launch_m(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                     cudaStream_t stream) {
  using C = Cfg<DQK, DV>;
  auto kern = paged_decode_kernel<DQK, DV, MOD>;
  static PerDeviceOnce once;
  const cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); });
  if (e != cudaSuccess) return e;
  if constexpr (MOD == kModRelBias) return launch_early(kern, dim3(ctas), kThreads, C::SMEM, stream, tq, tk, tv, a);
  kern<<<ctas, kThreads, C::SMEM, stream>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

template <int DQK, int DV>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                     cudaStream_t stream) {
  return a.score_mod == kModRelBias ? launch_m<DQK, DV, kModRelBias>(tq, tk, tv, a, ctas, stream)
                                    : launch_m<DQK, DV, kModNone>(tq, tk, tv, a, ctas, stream);
}

}  // namespace decode
}  // namespace paged

cudaError_t launch_paged_decode(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedArgs& a, int ctas, cudaStream_t stream) {
  if (d_qk == 64 && d_v == 64) return paged::decode::launch_d<64, 64>(tq, tk, tv, a, ctas, stream);
  if (d_qk == 128 && d_v == 128) return paged::decode::launch_d<128, 128>(tq, tk, tv, a, ctas, stream);
  if (d_qk == 192 && d_v == 128) return paged::decode::launch_d<192, 128>(tq, tk, tv, a, ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
