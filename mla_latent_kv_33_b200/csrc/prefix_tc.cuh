// Attention of a whole batch over one shared prefix on sm_100a tensor cores.
//
// The prefix's per-head keys and values are decompressed once (MLA
// walk-through, section 3 order A: K_h,i = [W_UK_h c_KV_i ; k_R,i], V_h,i =
// W_UV_h c_KV_i) and kept by the caller; every step then computes, for all T
// token rows t of the batch and every head h,
//   s_i = scale * qa[t][h] . K_h,i,  p = softmax_i(s),  o_P = sum_i p_i V_h,i,  i < P,
// and k_merge_shared joins o_P with the row's own suffix (mla_decode's absorbed
// attention, then W_UV) by the log-sum-exps of the two.
//
// Why order A here, when a decode step is absorbed otherwise: an absorbed
// (row, token) pair costs 2 * 128 * (576 + 512) = 278,528 flop and 1152 bytes
// that one row reads; an expanded one 2 * 128 * (192 + 128) = 81,920 flop, and
// its 65,664 bytes are read once for all rows of the batch. From a few dozen
// rows on the second is cheaper in both.
//
// Layout: one persistent CTA per SM. The 128-key tiles of all (block of 128
// token rows, head) pairs are laid end to end, row block outermost, and cut
// into equal ranges, one per CTA; a pair cut by a range boundary leaves fp32
// partials. (Row blocks outermost: the CTAs of two row blocks then walk the
// same heads at the same time and share K and V through L2.) Per CTA:
//   warps 0, 2, 3  TMA loads: K_C, V, k_R + Q (loads issued by one warp complete
//                  one after another, so they are spread over three)
//   warp 1         MMAs: S = Q K^T (M = 128 rows, N = 128 keys, K = 192), O += P V
//   warps 4-7, 8-11  two softmax groups: tile g of the CTA belongs to group
//                  g mod 2, which has its own score buffer, running maximum,
//                  sum and O accumulator, so that one group's exponentials run
//                  beside the other group's MMAs; at the end of a piece the two
//                  states are joined (thread = row in both groups).
// Tensor memory: S0, S1, O0, O1, 128 columns each. P is written in bf16 over
// its scores and read as the A operand of P V; V is an MN-major B operand.
// Rows past T and keys past P load as zeros (TMA), the keys are masked.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace pfx {

constexpr int DQK = 192, DV = 128, KTILE = 128, QROWS = 128, HEADS = 128;
constexpr int NUM_THREADS = 384, WARP_K = 0, WARP_MMA = 1, WARP_V = 2, WARP_R = 3, WARP_SMX = 4;
constexpr int CHUNK = 128 * 128;    // 128 rows x 64 columns bf16 (one swizzle-128 column)
constexpr int Q_BYTES = 3 * CHUNK;  // 48 KB
constexpr int K_BYTES = 3 * CHUNK;  // 48 KB: K_C chunks 0, 1 and the k_R chunk
constexpr int V_BYTES = 2 * CHUNK;  // 32 KB
constexpr int OFF_Q = 0, OFF_K = Q_BYTES, OFF_V = OFF_K + 2 * K_BYTES, OFF_ML = OFF_V + 2 * V_BYTES,
              OFF_BAR = OFF_ML + 2 * QROWS * 8;
// K slot s is released by the commit that completes S of the tile in it
constexpr int BAR_QF = 0, BAR_QE = 1, BAR_KF = 2, BAR_VF = 4, BAR_VE = 6, BAR_S = 8, BAR_P = 10, BAR_O = 12,
              BAR_OE = 13, NUM_BARS = 14;
constexpr int SMEM_BYTES = OFF_BAR + 8 * NUM_BARS + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "prefix attention shared memory budget");
constexpr uint32_t IDESC_S = idesc_bf16(QROWS, KTILE, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16(QROWS, DV, false, true);
constexpr int S_COL = 0, O_COL = 256;
constexpr float RESCALE_LOG2 = 8.f;

struct Params {
  int32_t T, P, nt, units;  // token rows, prefix length, key tiles, (row block, head) pairs
  int32_t part_rows;        // rows of a partial: min(T, 128)
  float scale, scale_log2;
  float *part_o;            // [units + CTAs][part_rows][128]
  float *part_lse;          // [units + CTAs][part_rows]
  const __nv_bfloat16 *qa;  // [T][n_h][192]
  __nv_bfloat16 *q;         // [T][n_h][576]: receives q_R in its last 64 columns
};

// First tile of CTA c's range when G CTAs share the tile line. The launch has
// at most as many CTAs as tiles, so no range is empty (unless the line is).
__host__ __device__ __forceinline__ int64_t range_start(int64_t tiles, int c, int G) { return tiles * c / G; }

struct Piece {
  int unit, t0, n;  // (row block, head) pair, first key tile, tiles
};
struct PieceIter {
  int64_t g, end;
  int nt;
  __device__ __forceinline__ bool next(Piece &pc) {
    if (g >= end) return false;
    pc.unit = static_cast<int>(g / nt);
    pc.t0 = static_cast<int>(g - static_cast<int64_t>(pc.unit) * nt);
    const int64_t left = end - g;
    pc.n = nt - pc.t0 < left ? nt - pc.t0 : static_cast<int>(left);
    g += pc.n;
    return true;
  }
};

__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_prefix_attend(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kc,
                    const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = sbase + OFF_BAR;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_BAR + 8 * NUM_BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int64_t line = static_cast<int64_t>(p.units) * p.nt;
  PieceIter it{range_start(line, blockIdx.x, gridDim.x), range_start(line, blockIdx.x + 1, gridDim.x), p.nt};

  if (threadIdx.x == 0) {
    for (int i = 0; i < NUM_BARS; ++i)
      mbar_init(bar(i), i == BAR_P || i == BAR_P + 1 ? 4 : (i == BAR_OE ? 8 : 1));
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == WARP_MMA) tmem_alloc<1>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();  // queries, keys and values may come from the kernel ahead on the stream
  Piece pc;

  if (warp == WARP_K || warp == WARP_V || warp == WARP_R) {
    // ----------------------------------------------------------- producers
    // Each warp waits for the slot it fills to be free; warp 0 arms the K slot
    // for its own boxes and for warp 3's.
    if (lane == 0) {
      int g = 0, npc = 0;
      bool ok = true;
      while (ok && it.next(pc)) {
        const int h = pc.unit % HEADS, r0 = pc.unit / HEADS * QROWS;
        if (warp == WARP_R) {
          if (npc > 0 && !mbar_wait(bar(BAR_QE), (npc - 1) & 1, abort_flag)) break;
          mbar_arrive_expect_tx(bar(BAR_QF), Q_BYTES);
          for (int c = 0; c < 3; ++c) tma_load_3d(sbase + OFF_Q + c * CHUNK, &tm_q, 64 * c, h, r0, bar(BAR_QF));
        }
        for (int i = 0; i < pc.n; ++i, ++g) {
          const int s = g & 1, use = g >> 1, key0 = (pc.t0 + i) * KTILE;
          if (use > 0 && !(ok = mbar_wait(bar((warp == WARP_V ? BAR_VE : BAR_S) + s), (use - 1) & 1, abort_flag))) break;
          const uint32_t kd = sbase + OFF_K + s * K_BYTES, vd = sbase + OFF_V + s * V_BYTES;
          if (warp == WARP_K) {
            mbar_arrive_expect_tx(bar(BAR_KF + s), K_BYTES);
            for (int c = 0; c < 2; ++c) tma_load_3d(kd + c * CHUNK, &tm_kc, 64 * c, key0, h, bar(BAR_KF + s));
          } else if (warp == WARP_R) {
            tma_load_2d(kd + 2 * CHUNK, &tm_kr, 0, key0, bar(BAR_KF + s));
          } else {
            mbar_arrive_expect_tx(bar(BAR_VF + s), V_BYTES);
            for (int c = 0; c < 2; ++c) tma_load_3d(vd + c * CHUNK, &tm_v, 64 * c, key0, h, bar(BAR_VF + s));
          }
        }
        ++npc;
      }
      // drain: the releases of the last use of each slot this warp fills have arrived
      for (int e = g - 2 > 0 ? g - 2 : 0; ok && e < g; ++e)
        ok = mbar_wait(bar((warp == WARP_V ? BAR_VE : BAR_S) + (e & 1)), (e >> 1) & 1, abort_flag);
      if (ok && warp == WARP_R && npc > 0) mbar_wait(bar(BAR_QE), (npc - 1) & 1, abort_flag);
    }
  } else if (warp == WARP_MMA) {
    // ---------------------------------------------------------- MMA issuer
    // QK of tile g + 1 goes out before PV of tile g; S of tile g overwrites P
    // of tile g - 2, whose PV was issued before it.
    if (lane == 0) {
      int g = 0, npc = 0;
      bool ok = true;
      const uint64_t dq = sdesc_sw128(sbase + OFF_Q, 16, 1024);
      auto pv = [&](int gt, bool first) -> bool {  // first: this piece's first tile of its group
        const int s = gt & 1;
        if (!mbar_wait(bar(BAR_VF + s), (gt >> 1) & 1, abort_flag)) return false;
        if (!mbar_wait(bar(BAR_P + s), (gt >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dv = sdesc_sw128(sbase + OFF_V + s * V_BYTES, CHUNK, 1024);
#pragma unroll
        for (int m = 0; m < KTILE / 16; ++m)
          tc_mma_ts<1>(tmem + O_COL + 128 * s, tmem + S_COL + 128 * s + 8 * m, sdesc_advance(dv, m * 2048), IDESC_PV,
                       (!first || m > 0) ? 1u : 0u);
        tc_commit(bar(BAR_VE + s));
        return true;
      };
      while (ok && it.next(pc)) {
        if (!mbar_wait(bar(BAR_QF), npc & 1, abort_flag)) break;
        for (int i = 0; i < pc.n; ++i, ++g) {
          const int s = g & 1;
          if (!(ok = mbar_wait(bar(BAR_KF + s), (g >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          const uint64_t dk = sdesc_sw128(sbase + OFF_K + s * K_BYTES, 16, 1024);
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma<1>(tmem + S_COL + 128 * s, sdesc_advance(dq, c * CHUNK + kk * 32),
                        sdesc_advance(dk, c * CHUNK + kk * 32), IDESC_S, (c > 0 || kk > 0) ? 1u : 0u);
          tc_commit(bar(BAR_S + s));
          if (i == pc.n - 1) tc_commit(bar(BAR_QE));
          if (i == 0) {
            // both O accumulators have been read out by the previous piece's epilogue
            if (npc > 0 && !(ok = mbar_wait(bar(BAR_OE), (npc - 1) & 1, abort_flag))) break;
            tc_fence_after();
          } else if (!(ok = pv(g - 1, i <= 2))) {
            break;
          }
        }
        if (!ok || !(ok = pv(g - 1, pc.n <= 2))) break;
        tc_commit(bar(BAR_O));
        ++npc;
      }
    }
  } else {
    // ------------------------------------------------- softmax + epilogue
    // A failed wait does not break the loops: every warp keeps the same
    // sequence of barriers and the error word reports it.
    const int grp = (warp - WARP_SMX) >> 2, sp = warp & 3;
    const int r = 32 * sp + lane;  // row of the block = tensor-memory lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * sp) << 16);
    const uint32_t s_addr = lane_addr + S_COL + 128 * grp, o_addr = lane_addr + O_COL + 128 * grp;
    float2 *ml = reinterpret_cast<float2 *>(smem + OFF_ML);  // [group][row]: running maximum and sum
    const float c2 = p.scale_log2;
    // q_R of every (row, head) into the absorbed queries' last columns, while the first tiles load
    {
      const int64_t n = static_cast<int64_t>(p.T) * HEADS * 8, stride = static_cast<int64_t>(gridDim.x) * 256;
      for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x - 128; e < n; e += stride) {
        const int64_t th = e >> 3;
        const int c = static_cast<int>(e & 7);
        *reinterpret_cast<uint4 *>(p.q + th * 576 + 512 + 8 * c) =
            *reinterpret_cast<const uint4 *>(p.qa + th * DQK + 128 + 8 * c);
      }
    }
    int g = 0, npc = 0;
    while (it.next(pc)) {
      float m_ref = -INFINITY, lsum = 0.f;
      const int g0 = g;
      g += pc.n;
      for (int gt = g0 + ((g0 ^ grp) & 1); gt < g; gt += 2) {
        mbar_wait_warp(bar(BAR_S + grp), (gt >> 1) & 1, abort_flag);
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld32(s_addr + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
        tmem_ld32(s_addr + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
        tmem_wait_ld();
        const int valid = p.P - (pc.t0 + gt - g0) * KTILE;  // keys of this tile inside the prefix (>= 1)
        if (valid < KTILE) {
#pragma unroll
          for (int c = 0; c < KTILE; ++c)
            if (c >= valid) sr[c] = __float_as_uint(-INFINITY);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < KTILE; ++c) mx = fmaxf(mx, __uint_as_float(sr[c]));
        if (gt - g0 < 2) {
          m_ref = mx;  // the group's first tile of this piece: PV overwrites O
        } else {
          // O and the sum are rescaled only when the maximum has grown by more
          // than 2^8: until then p stays below 2^8, far from overflow
          const bool need = (mx - m_ref) * c2 > RESCALE_LOG2;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx((m_ref - mx) * c2) : 1.f;
            if (need) m_ref = mx;
            lsum *= alpha;
            // S of this tile is complete, so the PV issued before it is too
#pragma unroll 1
            for (int q4 = 0; q4 < 8; ++q4) {
              uint32_t o[16];
              tmem_ld16(o_addr + 16 * q4, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(o_addr + 16 * q4, o);
            }
          }
        }
        const float mo = m_ref * c2;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          uint32_t pw[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(sr[64 * q4 + 2 * c]), c2, -mo));
            const float p1 = ex2_approx(fmaf(__uint_as_float(sr[64 * q4 + 2 * c + 1]), c2, -mo));
            ps[c & 3] += p0 + p1;
            pw[c] = pack_bf16x2(p0, p1);  // P is a tensor-core operand: one rounding to bf16
          }
          tmem_st32(s_addr + 32 * q4, pw);
        }
        tmem_wait_st();
        lsum += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_P + grp));
      }
      // ---- end of the piece: join the two groups' states, write the partial
      mbar_wait_warp(bar(BAR_O), npc & 1, abort_flag);
      tc_fence_after();
      ml[grp * QROWS + r] = make_float2(m_ref, lsum);
      named_bar_sync(1, 256);
      const float2 a = ml[r], b = ml[QROWS + r];
      const float M = fmaxf(a.x, b.x);
      const float wa = ex2_approx((a.x - M) * c2), wb = ex2_approx((b.x - M) * c2);  // 0 for a group without tiles
      const float L = a.y * wa + b.y * wb, inv = 1.f / L;
      const bool two = pc.n > 1;  // else only group g0 mod 2 has a (fresh) accumulator
      const int first = g0 & 1;
      const float w1 = (first ? wb : wa) * inv, w2 = (first ? wa : wb) * inv;
      const uint32_t o1 = lane_addr + O_COL + 128 * first, o2 = lane_addr + O_COL + 128 * (first ^ 1);
      const int t = pc.unit / HEADS * QROWS + r;
      const int64_t slot = static_cast<int64_t>(pc.unit) + blockIdx.x;
      float *dst = p.part_o + (slot * p.part_rows + r) * DV;
#pragma unroll 1
      for (int q4 = 0; q4 < 2; ++q4) {  // each group stores half of the columns
        const int col = 64 * grp + 32 * q4;
        uint32_t x[32], y[32];
        tmem_ld32(o1 + col, x);
        if (two) tmem_ld32(o2 + col, y);
        tmem_wait_ld();
        if (t < p.T) {
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = __uint_as_float(x[c + e]) * w1 + (two ? __uint_as_float(y[c + e]) * w2 : 0.f);
            *reinterpret_cast<float4 *>(dst + col + c) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (grp == 0 && t < p.T) p.part_lse[slot * p.part_rows + r] = M * p.scale + logf(L);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_OE));
      ++npc;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == WARP_MMA) tmem_dealloc<1>(tmem, 512);
}

// o[t][h] = (sum_k e^(lse_k) o_k) / sum_k e^(lse_k) over the prefix partials of
// (t, h) (normalised fp32) and its suffix readout (bf16 o_s, lse_s); lse = log
// sum_k e^(lse_k). One warp per (t, h), lane l the columns 4 l .. 4 l + 3, two
// partials per round trip. A sequence with a bad length is left unwritten.
struct MergeParams {
  int32_t T, n_q, P, nt, units, part_rows, ctas;
  int64_t capacity;
  const int32_t *seq_lens;
  const float *part_o, *part_lse;
  const __nv_bfloat16 *o_s;  // [T][n_h][128]
  const float *lse_s;        // [T][n_h]
  __nv_bfloat16 *o;          // [T][n_h][128]
  float *lse;                // [T][n_h] or NULL
};

__global__ void __launch_bounds__(256) k_merge_shared(const MergeParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int64_t th = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (th >= static_cast<int64_t>(p.T) * HEADS) return;
  const int t = static_cast<int>(th / HEADS), h = static_cast<int>(th % HEADS);
  const int32_t len = p.seq_lens[t / p.n_q];
  if (static_cast<int64_t>(len) < static_cast<int64_t>(p.P) + p.n_q || len > p.capacity) return;
  const uint2 sw = *reinterpret_cast<const uint2 *>(p.o_s + th * DV + 4 * lane);
  const __nv_bfloat162 s01 = *reinterpret_cast<const __nv_bfloat162 *>(&sw.x);
  const __nv_bfloat162 s23 = *reinterpret_cast<const __nv_bfloat162 *>(&sw.y);
  float4 acc = make_float4(__low2float(s01), __high2float(s01), __low2float(s23), __high2float(s23));
  float M = p.lse_s[th], Z = 1.f;
  const int unit = t / QROWS * HEADS + h, r = t % QROWS;
  // CTAs whose ranges hold the unit's tiles [a, e)
  const int64_t line = static_cast<int64_t>(p.units) * p.nt, a = static_cast<int64_t>(unit) * p.nt, e = a + p.nt;
  int k0 = 0, np = 0;
  if (p.nt > 0) {
    k0 = static_cast<int>(a * p.ctas / line);
    while (range_start(line, k0 + 1, p.ctas) <= a) ++k0;
    int k1 = k0;
    while (range_start(line, k1 + 1, p.ctas) < e) ++k1;
    np = k1 - k0 + 1;
  }
  for (int k = 0; k < np; k += 2) {
    const bool pair = k + 1 < np;
    const int64_t s0 = (static_cast<int64_t>(unit) + k0 + k) * p.part_rows + r, s1 = s0 + (pair ? p.part_rows : 0);
    const float l0 = __ldcg(p.part_lse + s0), l1 = pair ? __ldcg(p.part_lse + s1) : -INFINITY;
    const float4 x0 = __ldcg(reinterpret_cast<const float4 *>(p.part_o + s0 * DV) + lane);
    const float4 x1 = __ldcg(reinterpret_cast<const float4 *>(p.part_o + s1 * DV) + lane);
    const float Mn = fmaxf(M, fmaxf(l0, l1));
    const float w = __expf(M - Mn), w0 = __expf(l0 - Mn), w1 = __expf(l1 - Mn);
    Z = Z * w + w0 + w1;
    acc.x = acc.x * w + x0.x * w0 + x1.x * w1;
    acc.y = acc.y * w + x0.y * w0 + x1.y * w1;
    acc.z = acc.z * w + x0.z * w0 + x1.z * w1;
    acc.w = acc.w * w + x0.w * w0 + x1.w * w1;
    M = Mn;
  }
  const float inv = 1.f / Z;
  *reinterpret_cast<uint2 *>(p.o + th * DV + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[th] = M + logf(Z);
}

}  // namespace pfx
}  // namespace mla
