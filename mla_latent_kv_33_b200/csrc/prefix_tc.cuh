// Shared-prefix decode on sm_100a tensor cores: attention of a whole batch over
// one expanded prefix, and the join with each row's own suffix.
//
// The prefix's per-head keys and values are decompressed once (MLA
// walk-through, section 3 order A: K_h,i = [W_UK_h c_KV_i ; k_R,i], V_h,i =
// W_UV_h c_KV_i) and kept by the caller. A step is then four launches:
//   k_prefix_attend  for all T token rows t and heads h,
//                      s_i = scale * qa[t][h] . K_h,i,  o_P = sum_i softmax_i(s) V_h,i,  i < P,
//                    and, from the same queries in shared memory, the absorbed
//                    query q_lat,h = W_UK_h^T q_C,h (section 3 order B);
//   k_decode<., true>, k_combine   the suffix: absorbed attention to positions P ..;
//   k_shared_out     o_S,h = W_UV_h o_lat,h, joined with o_P by the log-sum-exps.
//
// Why order A for the prefix, when a decode step is absorbed otherwise: an
// absorbed (row, token) pair costs 2 * 128 * (576 + 512) = 278,528 flop and
// 1152 bytes that one row reads; an expanded one 2 * 128 * (192 + 128) = 81,920
// flop, and its 65,664 bytes are read once for all rows of the batch. Against
// the ordinary decode over shared pages the call is equal at about 64 rows over
// 4096 positions and 2.9 times as fast at 256 rows over 16384 (402 against 1175
// us), 2.4 times with the queries of either counted.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace pfx {

constexpr int DQK = 192, DV = 128, DC = 512, D = 576, KTILE = 128, QROWS = 128, HEADS = 128;
constexpr int ABS = DC / 128;  // absorb tiles of a unit: 128 columns of q_lat each
constexpr int NUM_THREADS = 384, WARP_K = 0, WARP_MMA = 1, WARP_V = 2, WARP_R = 3, WARP_SMX = 4;
constexpr int CHUNK = 128 * 128;    // 128 rows x 64 columns bf16 (one swizzle-128 column)
constexpr int Q_BYTES = 3 * CHUNK;  // 48 KB
// CG CTAs share a key tile: each holds 128 / CG keys of K and 128 / CG columns of V
template <int CG>
struct Cfg {
  static constexpr int STAGES = 2 * CG, K_CHUNK = CHUNK / CG, K_BYTES = 3 * K_CHUNK, V_BYTES = 2 * CHUNK / CG;
};
constexpr int OFF_Q = 0, OFF_K = Q_BYTES, OFF_V = OFF_K + 2 * 3 * CHUNK, OFF_STG = OFF_V + 2 * 2 * CHUNK;
constexpr int STG_WARP = 2048;  // per softmax warp: 32 rows x 64 bytes, to turn rows into wide stores
constexpr int OFF_MREF = OFF_STG + 8 * STG_WARP, OFF_BAR = OFF_MREF + QROWS * 4;
constexpr int SBUF = 3;  // score buffers
constexpr int BAR_QF = 0, BAR_QE = 1, BAR_KF = 2, BAR_KE = 6, BAR_VF = 10, BAR_VE = 14, BAR_S = 18, BAR_P = 21, BAR_O = 24,
              BAR_OE = 25, BAR_EXIT = 26, NUM_BARS = 27;
constexpr int SMEM_BYTES = OFF_BAR + 8 * NUM_BARS + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "prefix attention shared memory budget");
static_assert(2 * QROWS * 8 <= 8 * STG_WARP, "the groups' running maxima and sums alias the staging rows");
constexpr int S_COL = 0, O_COL = 128 * SBUF;
constexpr float RESCALE_LOG2 = 8.f;

struct Params {
  int32_t T, P, nt, units;  // token rows, prefix length, key tiles, (row group, head) pairs
  int32_t part_rows;        // rows of a partial: min(T, 128 CG)
  float scale, scale_log2;
  float *part_o;            // [units + clusters][part_rows][128]
  float *part_lse;          // [units + clusters][part_rows]
  const __nv_bfloat16 *qa;  // [T][n_h][192]
  __nv_bfloat16 *q;         // [T][n_h][576] = [q_lat | q_R]
  __nv_bfloat16 *q_lo;      // [T][n_h][512] = what rounding took from q_lat, or NULL
};

// First tile of cluster c's range when G clusters share the tile line. The
// launch has at most as many clusters as tiles, so no range is empty.
__host__ __device__ __forceinline__ int64_t range_start(int64_t tiles, int c, int G) { return tiles * c / G; }

struct Piece {
  int unit, t0, n;  // (row group, head) pair, first tile (ABS absorb tiles, then the key tiles), tiles
  __device__ __forceinline__ int keys_from() const { return t0 > ABS ? 0 : (ABS - t0 < n ? ABS - t0 : n); }
};
struct PieceIter {
  int64_t g, end;
  int per;  // tiles of a unit
  __device__ __forceinline__ bool next(Piece &pc) {
    if (g >= end) return false;
    pc.unit = static_cast<int>(g / per);
    pc.t0 = static_cast<int>(g - static_cast<int64_t>(pc.unit) * per);
    const int64_t left = end - g;
    pc.n = per - pc.t0 < left ? per - pc.t0 : static_cast<int>(left);
    g += pc.n;
    return true;
  }
};

// Each warp's 32 rows x 64 bytes, one row per lane as four 16-byte words, to
// words for row-contiguous stores: word k of row r sits at k ^ ((r >> 1) & 3),
// free of bank conflicts both ways. Lane l gets word l & 3 of rows l >> 2, + 8, + 16, + 24.
__device__ __forceinline__ void turn_rows(uint4 *stg, int lane, const uint4 (&in)[4], uint4 (&out)[4]) {
  const int sw = (lane >> 1) & 3;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) stg[4 * lane + (k ^ sw)] = in[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = (lane >> 2) + 8 * k;
    out[k] = stg[4 * r + ((lane & 3) ^ ((r >> 1) & 3))];
  }
}

// Layout: persistent CTAs, one per SM. The tiles of all (group of 128 CG token
// rows, head) units (four absorb tiles, then the 128-key tiles) are laid end to
// end, row group outermost, and cut into equal ranges; a unit cut by a range
// boundary leaves fp32 partials. Row groups outermost: the clusters of two row
// groups then walk the same heads at the same time and share K and V in L2.
//
// CG = 1 (T <= 128): one CTA per range. CG = 2 (more rows): a pair of SMs takes
// 256 rows, 128 each, with M = 256 pair MMAs; each CTA loads half of every tile
// (64 keys of K, 64 columns of V). On one SM, an M128 N128 MMA with both
// operands in shared memory runs at its full 64 clocks and reads 128 bytes per
// clock, all that shared memory gives, so that the loads' writes (80 KB per
// tile) and the MMAs slow each other; the pair halves the writes and the B
// reads. Measured (256 rows over 16384 positions, the whole call): 387 us with
// pairs, 436 with two single-CTA row groups.
//
// Bound: for up to 128 rows the reads of K_C and V (8192 positions: 103 us for
// 568 MB read and 39 MB written, of which 36 are absorbed queries and their
// remainders; 0.91 of the measured HBM rate, tensor pipe 43.5 % active); above,
// the MMAs (16384 positions, 256 rows: 265 us, tensor pipe 70 % active at the 1.6
// GHz that the power cap leaves; 1660 clocks per tile of a pair against 1282 of
// MMAs).
//
// Roles: warps 0, 2, 3 TMA loads (K_C; V and W_UK; Q and k_R: the loads one
// warp issues complete one after another, so they are spread over three), warp
// 1 MMAs (S = Q K^T, K = 192; O += P V; q_lat = q_C W_UK), warps 4-7 and 8-11
// two softmax groups, thread = row: tile g belongs to group g mod 2 and score
// buffer g mod 3, so that two tiles' exponentials run side by side and the
// scores of the tile two ahead are formed meanwhile. (With a buffer and an O
// accumulator per group instead, a group waits for its own P V and the next
// scores after every tile: 317 against 294 us for 256 rows over 16384
// positions.) The groups share one accumulator, so they share a row's reference
// maximum: after the maximum of its tile a group takes the reference over from
// the other, passes it on, and only then forms its exponentials. Tensor memory:
// three score buffers and O, 128 columns each. P is written in bf16 over its
// scores and read as the A operand of P V; V and W_UK are MN-major B operands.
// Rows past T and keys past P load as zeros (TMA), the keys are masked.
template <int CG>
__global__ void __launch_bounds__(NUM_THREADS, 1) __cluster_dims__(CG, 1, 1)
    k_prefix_attend(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kc,
                    const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_uk, const Params p) {
  using C = Cfg<CG>;
  constexpr uint32_t IDESC_S = idesc_bf16(QROWS * CG, KTILE, false, false);
  constexpr uint32_t IDESC_V = idesc_bf16(QROWS * CG, DV, false, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t rank = CG == 2 ? warp_uniform(cluster_ctarank()) : 0;
  const int warp = static_cast<int>(warp_uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int cluster = blockIdx.x / CG, nclusters = gridDim.x / CG;
  const uint32_t bars = sbase + OFF_BAR;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  auto lead = [&](int i) { return CG == 1 || rank == 0 ? bar(i) : mapa_shared(bar(i), 0); };  // the leader CTA's barrier
  auto commit = [&](int i) {  // to this barrier in every CTA of the cluster
    if constexpr (CG == 2) tc_commit_pair(bar(i), 0x3);
    else tc_commit(bar(i));
  };
  auto load2 = [&](uint32_t dst, const CUtensorMap *m, int x, int y, int b) {
    if constexpr (CG == 2) tma_load_2d_pair(dst, m, x, y, lead(b));
    else tma_load_2d(dst, m, x, y, bar(b));
  };
  auto load3 = [&](uint32_t dst, const CUtensorMap *m, int x, int y, int z, int b) {
    if constexpr (CG == 2) tma_load_3d_pair(dst, m, x, y, z, lead(b));
    else tma_load_3d(dst, m, x, y, z, bar(b));
  };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_BAR + 8 * NUM_BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int64_t line = static_cast<int64_t>(p.units) * (p.nt + ABS);
  PieceIter it{range_start(line, cluster, nclusters), range_start(line, cluster + 1, nclusters), p.nt + ABS};

  if (threadIdx.x == 0) {
    for (int i = 0; i < NUM_BARS; ++i)
      mbar_init(bar(i), i >= BAR_P && i < BAR_P + SBUF ? 4 * CG : (i == BAR_OE ? 8 * CG : 1));
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_uk);
  }
  if (warp == WARP_MMA) tmem_alloc<CG>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // barriers initialised and tensor memory allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();  // queries, keys and values may come from the kernel ahead on the stream
  Piece pc;

  if (warp < WARP_SMX) {
    reg_dec<120>();
    if (warp != WARP_MMA) {
      // --------------------------------------------------------- producers
      // K slots turn with the key tiles, V slots with all tiles (an absorb tile's
      // W_UK block takes a V slot). Each warp waits for the slot it fills to be
      // free; the leader's warps arm the barriers for both CTAs' boxes, warp 0
      // the K slot for its own boxes and for warp 3's.
      if (lane == 0) {
        int g = 0, gk = 0, npc = 0;
        bool ok = true;
        while (ok && it.next(pc)) {
          const int h = pc.unit % HEADS, r0 = pc.unit / HEADS * (QROWS * CG) + QROWS * static_cast<int>(rank);
          if (warp == WARP_R) {
            if (npc > 0 && !mbar_wait(bar(BAR_QE), (npc - 1) & 1, abort_flag)) break;
            if (rank == 0) mbar_arrive_expect_tx(bar(BAR_QF), CG * Q_BYTES);
            for (int c = 0; c < 3; ++c) load3(sbase + OFF_Q + c * CHUNK, &tm_q, 64 * c, h, r0, BAR_QF);
          }
          for (int i = 0; i < pc.n; ++i, ++g) {
            const int tt = pc.t0 + i, key0 = (tt - ABS) * KTILE;
            if (warp == WARP_V) {
              const int s = g % C::STAGES, use = g / C::STAGES;
              if (use > 0 && !(ok = mbar_wait(bar(BAR_VE + s), (use - 1) & 1, abort_flag))) break;
              if (rank == 0) mbar_arrive_expect_tx(bar(BAR_VF + s), CG * C::V_BYTES);
              const uint32_t vd = sbase + OFF_V + s * C::V_BYTES;
              for (int c = 0; c < 2 / CG; ++c) {
                const int col = 64 * (c + static_cast<int>(rank));
                if (tt < ABS) load2(vd + c * CHUNK, &tm_uk, 128 * tt + col, h * 128, BAR_VF + s);
                else load3(vd + c * CHUNK, &tm_v, col, key0, h, BAR_VF + s);
              }
            } else if (tt >= ABS) {
              const int s = gk % C::STAGES, use = gk / C::STAGES;
              if (use > 0 && !(ok = mbar_wait(bar(BAR_KE + s), (use - 1) & 1, abort_flag))) break;
              const uint32_t kd = sbase + OFF_K + s * C::K_BYTES;
              const int row = key0 + KTILE / CG * static_cast<int>(rank);
              if (warp == WARP_K) {
                if (rank == 0) mbar_arrive_expect_tx(bar(BAR_KF + s), CG * C::K_BYTES);
                for (int c = 0; c < 2; ++c) load3(kd + c * C::K_CHUNK, &tm_kc, 64 * c, row, h, BAR_KF + s);
              } else {
                load2(kd + 2 * C::K_CHUNK, &tm_kr, 0, row, BAR_KF + s);
              }
              ++gk;
            }
          }
          ++npc;
        }
        // drain: the releases of the last use of each slot this warp fills have arrived
        const int uses = warp == WARP_V ? g : gk, eb = warp == WARP_V ? BAR_VE : BAR_KE;
        for (int e = uses > C::STAGES ? uses - C::STAGES : 0; ok && e < uses; ++e)
          ok = mbar_wait(bar(eb + e % C::STAGES), (e / C::STAGES) & 1, abort_flag);
        if (ok && warp == WARP_R && npc > 0) mbar_wait(bar(BAR_QE), (npc - 1) & 1, abort_flag);
      }
    } else if (rank == 0) {
      // -------------------------------------------------------- MMA issuer
      // (the whole warp, one elected lane issuing)
      // The scores of tile g + 2 go out before P V of tile g; they overwrite P of
      // tile g - 1, whose P V was issued before them.
      int g = 0, gk = 0, npc = 0, npk = 0;  // first tile of the piece, key tiles, pieces, pieces with key tiles
      const uint32_t tm = warp_uniform(tmem);
      const uint64_t dq = sdesc_sw128(sbase + OFF_Q, 16, 1024);
      auto issue = [&](int gt, bool absorb, bool last) -> bool {
        const uint32_t d = tm + S_COL + 128 * (gt % SBUF);
        if (absorb) {  // 128 columns of q_lat: K = the 128 columns of q_C
          const int vs = gt % C::STAGES;
          if (!mbar_wait_warp(bar(BAR_VF + vs), (gt / C::STAGES) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint64_t dw = sdesc_sw128(sbase + OFF_V + vs * C::V_BYTES, CHUNK, 1024);
          if (elect_one()) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
              tc_mma<CG>(d, sdesc_advance(dq, (m >> 2) * CHUNK + (m & 3) * 32), sdesc_advance(dw, m * 2048), IDESC_V,
                         m > 0 ? 1u : 0u);
            commit(BAR_VE + vs);
            commit(BAR_S + gt % SBUF);
            if (last) commit(BAR_QE);
          }
        } else {
          const int ks = gk % C::STAGES;
          if (!mbar_wait_warp(bar(BAR_KF + ks), (gk / C::STAGES) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint64_t dk = sdesc_sw128(sbase + OFF_K + ks * C::K_BYTES, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma<CG>(d, sdesc_advance(dq, c * CHUNK + kk * 32), sdesc_advance(dk, c * C::K_CHUNK + kk * 32), IDESC_S,
                           (c > 0 || kk > 0) ? 1u : 0u);
            commit(BAR_KE + ks);
            commit(BAR_S + gt % SBUF);
            if (last) commit(BAR_QE);
          }
          ++gk;
        }
        __syncwarp();
        return true;
      };
      // once tile gt's group has answered: P V of a key tile (ko: its place among
      // the piece's key tiles); an absorb tile's buffer is then free
      auto finish = [&](int gt, bool absorb, int ko) -> bool {
        const int b = gt % SBUF, vs = gt % C::STAGES;
        if (!absorb && !mbar_wait_warp(bar(BAR_VF + vs), (gt / C::STAGES) & 1, abort_flag)) return false;
        if (!mbar_wait_warp(bar(BAR_P + b), (gt / SBUF) & 1, abort_flag)) return false;
        if (absorb) return true;
        // O of the last piece has been read out
        if (ko == 0 && npk > 0 && !mbar_wait_warp(bar(BAR_OE), (npk - 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dv = sdesc_sw128(sbase + OFF_V + vs * C::V_BYTES, CHUNK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int m = 0; m < KTILE / 16; ++m)
            tc_mma_ts<CG>(tm + O_COL, tm + S_COL + 128 * b + 8 * m, sdesc_advance(dv, m * 2048), IDESC_V,
                          (ko > 0 || m > 0) ? 1u : 0u);
          commit(BAR_VE + vs);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      while (ok && it.next(pc)) {
        if (!mbar_wait_warp(bar(BAR_QF), npc & 1, abort_flag)) break;
        const int kf = pc.keys_from();
        for (int i = -2; i < pc.n && ok; ++i) {
          if (i + 2 < pc.n) ok = issue(g + i + 2, i + 2 < kf, i + 3 == pc.n);
          if (ok && i >= 0) ok = finish(g + i, i < kf, i - kf);
        }
        if (!ok) break;
        g += pc.n;
        if (kf < pc.n) {
          if (elect_one()) commit(BAR_O);
          __syncwarp();
          ++npk;
        }
        ++npc;
      }
    }
  } else {
    reg_inc<192>();
    // ------------------------------------------------- softmax + epilogue
    // A failed wait does not break the loops: every warp keeps the same
    // sequence of barriers and the error word reports it.
    const int grp = (warp - WARP_SMX) >> 2, sp = warp & 3;
    const int r = 32 * sp + lane;  // row of the CTA's block = tensor-memory lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * sp) << 16), o_addr = lane_addr + O_COL;
    // hand-over of the reference maxima between the two warps of the same rows
    float *mref = reinterpret_cast<float *>(smem + OFF_MREF);
    const uint32_t bar_take = 2 + 4 * (grp ^ 1) + sp, bar_give = 2 + 4 * grp + sp;
    float2 *ml = reinterpret_cast<float2 *>(smem + OFF_STG);  // [group][row]: running maximum and sum
    uint4 *stg = reinterpret_cast<uint4 *>(smem + OFF_STG + STG_WARP * (warp - WARP_SMX));
    const float c2 = p.scale_log2;
    auto arrive = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || rank == 0) mbar_arrive(bar(b));
        else mbar_arrive_cluster(mapa_shared(bar(b), 0));
      }
    };
    int g = 0, npk = 0;
    while (it.next(pc)) {
      const int h = pc.unit % HEADS, kf = pc.keys_from();
      // first row of this CTA's block, and the first of this warp's rows
      const int rb = pc.unit / HEADS * (QROWS * CG) + QROWS * static_cast<int>(rank), t0 = rb + 32 * sp;
      float m_ref = -INFINITY, lsum = 0.f;
      const int g0 = g;
      g += pc.n;
      for (int gt = g0 + ((g0 ^ grp) & 1); gt < g; gt += 2) {
        const int i = gt - g0, tt = pc.t0 + i, buf = gt % SBUF;
        const uint32_t s_addr = lane_addr + S_COL + 128 * buf;
        if (i < kf) {
          // ---- absorb tile: 128 columns of q_lat, rounded to bf16 (a tensor-core
          // operand of the suffix), the remainder kept for the lse of the result
          if (tt == 0) {  // q_R goes along: 8 lanes per row
            for (int k = 0; k < 8; ++k) {
              const int t = t0 + 4 * k + (lane >> 3), c = lane & 7;
              const int64_t th = static_cast<int64_t>(t) * HEADS + h;
              if (t < p.T)
                *reinterpret_cast<uint4 *>(p.q + th * D + DC + 8 * c) =
                    *reinterpret_cast<const uint4 *>(p.qa + th * DQK + DV + 8 * c);
            }
          }
          mbar_wait_warp(bar(BAR_S + buf), (gt / SBUF) & 1, abort_flag);
          tc_fence_after();
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t x[32];
            tmem_ld32(s_addr + 32 * q4, x);
            tmem_wait_ld();
            uint4 hi[4], lo[4], out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hw[4], lw[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(x[8 * k + 2 * e]), b = __uint_as_float(x[8 * k + 2 * e + 1]);
                const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
                hw[e] = *reinterpret_cast<const uint32_t *>(&v);
                lw[e] = pack_bf16x2(a - __low2float(v), b - __high2float(v));
              }
              hi[k] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
              lo[k] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            }
            const int col = 128 * tt + 32 * q4 + 8 * (lane & 3);
            turn_rows(stg, lane, hi, out);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int t = t0 + (lane >> 2) + 8 * k;
              if (t < p.T) *reinterpret_cast<uint4 *>(p.q + (static_cast<int64_t>(t) * HEADS + h) * D + col) = out[k];
            }
            if (p.q_lo != nullptr) {
              turn_rows(stg, lane, lo, out);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int t = t0 + (lane >> 2) + 8 * k;
                if (t < p.T) *reinterpret_cast<uint4 *>(p.q_lo + (static_cast<int64_t>(t) * HEADS + h) * DC + col) = out[k];
              }
            }
          }
          arrive(BAR_P + buf);
          continue;
        }
        // ---- key tile
        mbar_wait_warp(bar(BAR_S + buf), (gt / SBUF) & 1, abort_flag);
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld32(s_addr + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
        tmem_ld32(s_addr + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
        tmem_wait_ld();
        const int valid = p.P - (tt - ABS) * KTILE;  // keys of this tile inside the prefix (>= 1)
        if (valid < KTILE) {
#pragma unroll
          for (int c = 0; c < KTILE; ++c)
            if (c >= valid) sr[c] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < KTILE; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the reference maximum: that of the tile before, taken over from the other
        // group, unless this tile's maximum exceeds it by more than 2^8 (until then
        // p stays below 2^8, far from overflow); then O is rescaled
        float m_new = mt;
        if (i > kf) {
          named_bar_sync(bar_take, 64);
          m_new = mref[r];
          const bool need = (mt - m_new) * c2 > RESCALE_LOG2;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx((m_new - mt) * c2) : 1.f;
            if (need) m_new = mt;
            const int vs = (gt - 1) % C::STAGES;  // every P V so far has finished
            mbar_wait_warp(bar(BAR_VE + vs), ((gt - 1) / C::STAGES) & 1, abort_flag);
            tc_fence_after();
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
        if (i + 1 < pc.n) {
          mref[r] = m_new;
          named_bar_arrive(bar_give, 64);
        }
        lsum *= ex2_approx((m_ref - m_new) * c2);  // 1 unless the reference moved; 0 * 0 at first
        m_ref = m_new;
        const f32x2 scale2 = make_f32x2(c2, c2), shift2 = make_f32x2(-m_ref * c2, -m_ref * c2);
        f32x2 ps[2] = {make_f32x2(0.f, 0.f), make_f32x2(0.f, 0.f)};
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          uint32_t pw[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const f32x2 t =
                fma2(make_f32x2(__uint_as_float(sr[64 * q4 + 2 * c]), __uint_as_float(sr[64 * q4 + 2 * c + 1])), scale2, shift2);
            float2 e = split(t);
            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            ps[c & 1] = add2(ps[c & 1], make_f32x2(e.x, e.y));
            pw[c] = pack_bf16x2(e.x, e.y);  // P is a tensor-core operand: one rounding to bf16
          }
          tmem_st32(s_addr + 32 * q4, pw);
        }
        tmem_wait_st();
        const float2 sum = split(add2(ps[0], ps[1]));
        lsum += sum.x + sum.y;
        arrive(BAR_P + buf);
      }
      if (kf == pc.n) continue;  // absorb tiles only: no partial
      // ---- end of the piece: join the two groups' sums, write the partial
      mbar_wait_warp(bar(BAR_O), npk & 1, abort_flag);
      tc_fence_after();
      named_bar_sync(1, 256);  // the staging rows under ml are no longer read
      ml[grp * QROWS + r] = make_float2(m_ref, lsum);
      named_bar_sync(1, 256);
      const float2 a = ml[r], b = ml[QROWS + r];
      named_bar_sync(1, 256);
      const float M = fmaxf(a.x, b.x);  // the last reference; 0 weight for a group without key tiles
      const float L = a.y * ex2_approx((a.x - M) * c2) + b.y * ex2_approx((b.x - M) * c2), inv = 1.f / L;
      const int64_t slot = (static_cast<int64_t>(pc.unit) + cluster) * p.part_rows;
      const int pr = QROWS * static_cast<int>(rank);  // this CTA's first row of the partial
#pragma unroll 1
      for (int q4 = 0; q4 < 4; ++q4) {  // each group stores half of the columns, 16 at a time
        const int col = 64 * grp + 16 * q4;
        uint32_t x[16];
        tmem_ld16(o_addr + col, x);
        tmem_wait_ld();
        uint4 v[4], out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = make_uint4(__float_as_uint(__uint_as_float(x[4 * k]) * inv), __float_as_uint(__uint_as_float(x[4 * k + 1]) * inv),
                            __float_as_uint(__uint_as_float(x[4 * k + 2]) * inv), __float_as_uint(__uint_as_float(x[4 * k + 3]) * inv));
        turn_rows(stg, lane, v, out);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = 32 * sp + (lane >> 2) + 8 * k;
          if (rb + rr < p.T) *reinterpret_cast<uint4 *>(p.part_o + (slot + pr + rr) * DV + col + 4 * (lane & 3)) = out[k];
        }
      }
      if (grp == 0 && rb + r < p.T) p.part_lse[slot + pr + r] = M * p.scale + logf(L);
      arrive(BAR_OE);
      ++npk;
    }
  }
  // ---- teardown: the CTAs of a pair are done with each other's barriers, then free tensor memory
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    if (threadIdx.x == 0) {
      mbar_arrive_cluster(mapa_shared(bar(BAR_EXIT), rank ^ 1));
      mbar_wait(bar(BAR_EXIT), 0, nullptr);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == WARP_MMA) tmem_dealloc<CG>(tmem, 512);
}

// Suffix readout and join: for one (block of 128 token rows, head) per CTA,
//   o_S = W_UV_h o_lat,h  (M = 128 rows, N = 128, K = 512, fp32 in tensor memory),
//   o = (e^lse_S o_S + sum_k e^lse_k o_k) / (e^lse_S + sum_k e^lse_k)
// over the prefix partials o_k of the rows. o_S never leaves the SM, and is not
// rounded on the way; o_lat was, once, to be the operand here (as between
// mla_decode and mla_out_proj: rows that see mostly suffix end up to 0.0027 off,
// relative, of which the output's own rounding is 0.0017. A second operand with
// the remainder would read and write 2 x 33 MB more at 256 rows). Bound: the reads of o_lat, q_lo, W_UV and the partials
// (128 rows over 8192 positions: 68 MB from HBM in 18 us with cold caches).
//
// The scores of the suffix were formed with q_lat rounded to bf16 (a
// tensor-core operand), which is within the precision of o but not of an fp32
// lse: the rounding dq moves lse_S by scale * dq . o_lat (its gradient), so the
// returned lse adds that product back, formed here as the diagonal of a second
// 128 x 128 product of o_lat with q_lo.
namespace so {
constexpr int MAX_PARTS = 3;
constexpr int NUM_THREADS = 384, STAGE = 3 * CHUNK, BK = 64, KB = DC / BK;
constexpr int PITCH = DV + 4;  // floats per row of the staged o_S: conflict-free for 16-byte words
constexpr int MAX_STAGES = 4;
constexpr int smem_bytes(int stages) { return stages * STAGE + 8 * (2 * MAX_STAGES + 1) + 16 + 3 * 128 * 4 + 1024; }
static_assert(2 * STAGE >= QROWS * PITCH * 4, "o_S is staged over the pipeline's stages");
static_assert(2 * smem_bytes(2) <= 232448 && smem_bytes(MAX_STAGES) <= 232448, "suffix readout shared memory budget");
struct Params {
  int32_t T, n_q, P, nt, units, part_rows, clusters, group, stages;  // group: row blocks per prefix unit (CG)
  int64_t capacity;
  float scale;
  const int32_t *seq_lens;
  const float *part_o, *part_lse;
  const float *lse_s;  // [T][n_h]
  __nv_bfloat16 *o;    // [T][n_h][128]
  float *lse;          // [T][n_h] or NULL
};
}  // namespace so

template <int CTAS>  // per SM (registers for 8 or 4 rows' loads in flight per warp)
__global__ void __launch_bounds__(so::NUM_THREADS, CTAS)
    k_shared_out(const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_uv,
                 const __grid_constant__ CUtensorMap tm_lo, const so::Params p) {
  constexpr int RSTEP = CTAS == 1 ? 8 : 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = static_cast<int>(warp_uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int h = blockIdx.x % HEADS, blk = blockIdx.x / HEADS, t0 = blk * QROWS;
  uint8_t *misc = smem + p.stages * so::STAGE;
  const uint32_t bars = sbase + p.stages * so::STAGE;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (so::MAX_STAGES + s); };
  const uint32_t done = bars + 8u * (2 * so::MAX_STAGES);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 8 * (2 * so::MAX_STAGES + 1));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *diag = reinterpret_cast<float *>(misc + 8 * (2 * so::MAX_STAGES + 1) + 16);  // [128]
  const bool want_lse = p.lse != nullptr;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * so::MAX_STAGES + 1; ++i) mbar_init(bars + 8u * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 0 || warp == 2 || warp == 3) {
    // one warp per operand: o_lat (arms the stage), W_UV, q_lo. The first W_UV
    // boxes go out before the wait for the suffix decode (weights).
    if (warp != 2) griddep_wait();
    if (lane == 0 && (warp != 3 || want_lse)) {
      bool ok = true;
      for (int i = 0; i < so::KB && ok; ++i) {
        const int s = i % p.stages;
        const uint32_t dst = sbase + s * so::STAGE;
        if (i >= p.stages && !(ok = mbar_wait(empty(s), (i / p.stages - 1) & 1, abort_flag))) break;
        if (warp == 0) {
          mbar_arrive_expect_tx(full(s), (want_lse ? 3 : 2) * CHUNK);
          tma_load_3d(dst, &tm_o, so::BK * i, h, t0, full(s));
        } else if (warp == 2) {
          tma_load_2d(dst + CHUNK, &tm_uv, so::BK * i, h * DV, full(s));
        } else {
          tma_load_3d(dst + 2 * CHUNK, &tm_lo, so::BK * i, h, t0, full(s));
        }
      }
      // drain: the releases of the stages' last uses have arrived
      for (int i = so::KB - p.stages; ok && i < so::KB; ++i) ok = mbar_wait(empty(i % p.stages), (i / p.stages) & 1, abort_flag);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16(QROWS, DV, false, false);
    const uint32_t tm = warp_uniform(tmem);
    for (int i = 0; i < so::KB; ++i) {
      const int s = i % p.stages;
      if (!mbar_wait_warp(full(s), (i / p.stages) & 1, abort_flag)) break;
      tc_fence_after();
      const uint64_t da = sdesc_sw128(sbase + s * so::STAGE, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < so::BK / 16; ++kk) {
          const uint64_t a = sdesc_advance(da, kk * 32);
          tc_mma<1>(tm, a, sdesc_advance(a, CHUNK), idesc, (i > 0 || kk > 0) ? 1u : 0u);
          if (want_lse) tc_mma<1>(tm + 128, a, sdesc_advance(a, 2 * CHUNK), idesc, (i > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(empty(s));
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(done);
    __syncwarp();
  } else {
    griddep_wait();
    const int grp = (warp - 4) >> 2, sp = warp & 3, r = 32 * sp + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * sp) << 16);
    float *o_s = reinterpret_cast<float *>(smem);  // [128][PITCH], over the stages: every MMA has finished
    // the clusters whose ranges hold key tiles [a, e) of this block's unit
    const int unit = blk / p.group * HEADS + h;
    const int64_t per = p.nt + ABS, line = p.units * per, a = unit * per + ABS, e = (unit + 1) * per;
    int k0 = 0, np = 0;
    if (p.nt > 0) {
      k0 = static_cast<int>(a * p.clusters / line);
      while (range_start(line, k0 + 1, p.clusters) <= a) ++k0;
      int k1 = k0;
      while (range_start(line, k1 + 1, p.clusters) < e) ++k1;
      np = k1 - k0 + 1;
    }
    // This warp joins 16 rows. Lane l < 16 weighs row l's parts while the product
    // runs: w[k] for partial k (at most three clusters share a unit: there are at
    // most 3 / 2 as many clusters as units, so that a range holds more than half a
    // unit's tiles), ws for the suffix, normalised.
    const int row0 = 16 * (warp - 4);
    const int64_t pr0 = (static_cast<int64_t>(unit) + k0) * p.part_rows + blk % p.group * QROWS + row0;
    using so::MAX_PARTS;
    float w[MAX_PARTS] = {0.f, 0.f, 0.f}, ws = 0.f, ls = 0.f, M = 0.f, Zp = 0.f;
    bool valid = false;
    if (lane < 16 && t0 + row0 + lane < p.T) {
      const int t = t0 + row0 + lane;
      const int32_t len = p.seq_lens[t / p.n_q];
      valid = static_cast<int64_t>(len) >= static_cast<int64_t>(p.P) + p.n_q && len <= p.capacity;
      if (valid) {
        float l[MAX_PARTS];
        M = ls = p.lse_s[static_cast<int64_t>(t) * HEADS + h];
#pragma unroll
        for (int k = 0; k < MAX_PARTS; ++k) {
          l[k] = k < np ? __ldcg(p.part_lse + pr0 + lane + static_cast<int64_t>(k) * p.part_rows) : -INFINITY;
          M = fmaxf(M, l[k]);
        }
#pragma unroll
        for (int k = 0; k < MAX_PARTS; ++k) Zp += w[k] = __expf(l[k] - M);
        ws = __expf(ls - M);
        const float inv = 1.f / (Zp + ws);
        ws *= inv;
#pragma unroll
        for (int k = 0; k < MAX_PARTS; ++k) w[k] *= inv;
      }
    }
    const uint32_t rows_ok = __ballot_sync(0xffffffffu, valid);
    // the prefix's share of RSTEP rows, lane l the columns 4 l .. 4 l + 3; the
    // first ones before the product is done. All loads of a step go out together
    // (a partial past np is read at the last one's place, with weight 0).
    float4 acc[RSTEP];
    auto load_rows = [&](int i0) {
#pragma unroll
      for (int i = 0; i < RSTEP; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < np; k += 2) {
        const float *src = p.part_o + (pr0 + i0 + static_cast<int64_t>(k) * p.part_rows) * DV + 4 * lane;
        const int64_t next = k + 1 < np ? static_cast<int64_t>(p.part_rows) * DV : 0;
        const float wa = k == 0 ? w[0] : w[2], wb = k == 0 ? w[1] : 0.f;
        float4 x[RSTEP], y[RSTEP];
#pragma unroll
        for (int i = 0; i < RSTEP; ++i) {
          const bool ok = rows_ok >> (i0 + i) & 1;
          x[i] = ok ? __ldcg(reinterpret_cast<const float4 *>(src + i * DV)) : make_float4(0.f, 0.f, 0.f, 0.f);
          y[i] = ok ? __ldcg(reinterpret_cast<const float4 *>(src + next + i * DV)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < RSTEP; ++i) {
          const float w0 = __shfl_sync(0xffffffffu, wa, i0 + i), w1 = __shfl_sync(0xffffffffu, wb, i0 + i);
          acc[i].x += x[i].x * w0 + y[i].x * w1;
          acc[i].y += x[i].y * w0 + y[i].y * w1;
          acc[i].z += x[i].z * w0 + y[i].z * w1;
          acc[i].w += x[i].w * w0 + y[i].w * w1;
        }
      }
    };
    load_rows(0);
    mbar_wait_warp(done, 0, abort_flag);
    tc_fence_after();
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      uint32_t x[16];
      tmem_ld16(lane_addr + 64 * grp + 16 * q4, x);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4 *>(o_s + r * so::PITCH + 64 * grp + 16 * q4 + 4 * k) =
            make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    }
    if (grp == 0 && want_lse) {  // element (r, r) of the second product
      float dg = 0.f;
#pragma unroll
      for (int q4 = 0; q4 < 2; ++q4) {
        uint32_t x[16];
        tmem_ld16(lane_addr + 128 + 32 * sp + 16 * q4, x);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) dg = lane == 16 * q4 + c ? __uint_as_float(x[c]) : dg;
      }
      diag[r] = dg;
    }
    named_bar_sync(1, 256);
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += RSTEP) {
      if (i0 > 0) load_rows(i0);
#pragma unroll
      for (int i = 0; i < RSTEP; ++i) {
        const int rr = row0 + i0 + i;
        const float wsr = __shfl_sync(0xffffffffu, ws, i0 + i);
        if (!(rows_ok >> (i0 + i) & 1)) continue;
        const float4 x = *reinterpret_cast<const float4 *>(o_s + rr * so::PITCH + 4 * lane);
        *reinterpret_cast<uint2 *>(p.o + (static_cast<int64_t>(t0 + rr) * HEADS + h) * DV + 4 * lane) =
            make_uint2(pack_bf16x2(acc[i].x + x.x * wsr, acc[i].y + x.y * wsr),
                       pack_bf16x2(acc[i].z + x.z * wsr, acc[i].w + x.w * wsr));
      }
    }
    if (valid && want_lse)
      p.lse[static_cast<int64_t>(t0 + row0 + lane) * HEADS + h] =
          M + logf(Zp + __expf(ls + p.scale * diag[row0 + lane] - M));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, 256);
}

}  // namespace pfx
}  // namespace mla
