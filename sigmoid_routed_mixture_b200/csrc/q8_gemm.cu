// q8_gemm.cu -- products of 8-bit integers with a scale per row and per
// channel, dense or by expert groups, on the 5th-generation tensor cores:
//     y[r][n] = x_scale[r] * w_scale[g][n] * sum_k x[r][k] w[g][n][k] (+ residual[r][n])
// and, with the gate and up channels interleaved 16 + 16, h = silu(gate) * up.
// The sum is exact (tcgen05.mma kind::i8, int32 accumulators in tensor memory;
// K <= 65536, so |sum| <= 65536 * 128 * 128 = 2^30): the result depends on
// neither the tiling nor the order of the split reductions.
//
// Operand roles, tiles and barriers are those of the 16-bit grouped products
// (grouped_gemm.cu): the weights are the MMA's M side (128 rows per CTA, 256
// per CTA pair), the token rows its N side (a tile's rows rounded up to 32),
// both by TMA with 128-byte swizzling, K steps of 128 bytes = 128 elements,
// a persistent warp-specialised kernel, tiles dealt out by an atomic counter,
// token block fastest.  A k-block moves the bytes of a 16-bit one in the same
// MMA time and covers twice the K.
//
// Split reduction: where there are fewer tiles than CTAs (or pairs), each
// tile's K range is cut into equal parts, one a unit.  The epilogue warps of a
// part leave their int32 partial sums in the workspace and count themselves
// in, and the last of a tile's parts to arrive adds the others' sums to its own
// accumulator and finishes.  Nothing waits, and integer sums are exact in any
// order, so the result does not change from run to run.
//
// The counters return to zero by themselves (each wraps at its last arrival),
// so a call needs no clearing launch before it (1 to 3 us of a decode
// product).  The workspace's ready word says that they can be trusted: it is
// set when a workspace is initialised and taken back by a call that gave up a
// wait.  Without it the tiles are dealt out whole and in a fixed stride.
#include <cuda.h>

#include "kernels.h"
#include "launch.cuh"
#include "rowio.cuh"

namespace srm {

namespace q8 {
constexpr int BM = 128;           // weight rows per CTA (tensor-memory lanes)
constexpr int BK = 128;           // elements (bytes) of K per step: one swizzle atom
constexpr int EPI_WARPS = kQ8EpiWarps;
constexpr int SCHED_WARP = 2 + EPI_WARPS;
constexpr int THREADS = 32 * (SCHED_WARP + 1);
constexpr int MAX_GROUPS = kQ8MaxGroups;
constexpr int MAX_STAGES = 8;
constexpr int TILE_RING = 4;

template <bool kPair>
struct Cfg {
  static constexpr int BT = kPair ? kQ8PairRows : kQ8SoloRows;  // token rows per tile
  static constexpr int W_BLOCK = kPair ? 2 * BM : BM;
  static constexpr int TOK_ROWS = kPair ? BT / 2 : BT;
  static constexpr int STAGES = kPair ? 6 : 8;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = TOK_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr uint32_t TMEM_COLS = 2 * BT;
  static constexpr uint32_t EPI_ARRIVALS = (kPair ? 2 : 1) * EPI_WARPS;
  static constexpr int RANKS = kPair ? 2 : 1;
};

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tile_full[TILE_RING];
  uint64_t tile_empty[TILE_RING];
  alignas(16) int tile_ring[TILE_RING][4];  // g (-1: no more), first row, rows, first weight row
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint64_t draw;  // the producer is near the end of its tile: the next one is to be drawn
  uint32_t tmem_base;
  int abort_flag;
  int ready;
  int mma_consumed;
  int total_mtiles;
  int tile_start[MAX_GROUPS + 1];
  int grp_off[MAX_GROUPS + 1];
  alignas(16) float row_scale[EPI_WARPS][kQ8PairRows];  // each epilogue warp's copy of its tile's
};
template <bool kPair>
constexpr size_t smem_bytes() {
  return 1024 + Cfg<kPair>::STAGES * Cfg<kPair>::STAGE_BYTES + sizeof(Smem);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory above 227 KB");

// Instruction descriptor of kind::i8: int32 accumulator (2), signed operands
// (1), both K-major.  N is a multiple of 32, legal for single CTAs and pairs.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A box of a tensor map to shared memory, completion counted on the mbarrier at
// `bar` (the leader's, for a pair; no multicast).
template <bool kPair>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *tmap, uint32_t bar, int32_t c0,
                                          int32_t c1) {
  if (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

struct Tile {
  int g;         // group
  int row_base;  // first token row
  int rows;      // valid token rows
  int n;         // MMA N: rows rounded up to 32
  int w0;        // first weight row within the group
  int kb0, kb1;  // k-blocks of it to do here (all of them unless it is cut)
};

// Tiles in (group, weight block, token block) order, token block fastest
// (groups of more than m_chunk token blocks in chunks, each through all weight
// blocks).
template <bool kPair>
__device__ __forceinline__ Tile decode(const Smem &s, const Q8GemmArgs &p, int n_tiles, int m_chunk,
                                       int kblocks, int tile) {
  Tile c;
  c.kb0 = 0;
  c.kb1 = kblocks;
  const int mt_flat = tile / n_tiles;
  int lo = 0, hi = p.groups - 1;  // last g with tile_start[g] <= mt_flat
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tile_start[mid] <= mt_flat)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int mblocks = s.tile_start[lo + 1] - s.tile_start[lo];
  const int local = tile - s.tile_start[lo] * n_tiles;
  // (a group of at most m_chunk token blocks, the usual one, needs no division)
  const int m0 = mblocks <= m_chunk ? 0 : local / n_tiles / m_chunk * m_chunk;
  const int cm = min(m_chunk, mblocks - m0);  // token blocks in this chunk
  const int r = local - m0 * n_tiles;
  const int nt = r / cm;
  const int mt = m0 + (r - nt * cm);
  constexpr int BT = Cfg<kPair>::BT;
  c.g = lo;
  c.row_base = s.grp_off[lo] + mt * BT;
  c.rows = max(0, min(BT, s.grp_off[lo + 1] - c.row_base));
  c.n = max(32, (c.rows + 31) & ~31);
  c.w0 = nt * Cfg<kPair>::W_BLOCK;
  return c;
}

// The tile that the scheduler published in ring slot ts; false: no more.
__device__ __forceinline__ bool ring_tile(const Smem &s, uint32_t ts, int kblocks, Tile *c) {
  const volatile int *e = s.tile_ring[ts];
  c->g = e[0];
  c->row_base = e[1];
  c->rows = e[2];
  c->w0 = e[3];
  c->n = max(32, (c->rows + 31) & ~31);
  c->kb0 = 0;
  c->kb1 = kblocks;
  return c->g >= 0;
}

// Two results (of two rows) in their type.  fp16 saturates at +-65504, as the
// library's other fp16 intermediates do: an infinity becomes the largest finite
// number, `largest` keeps the largest magnitudes seen for the flag; NaN stays.
template <typename T>
struct Pair2 {
  T lo, hi;
};
template <typename T>
__device__ __forceinline__ Pair2<T> to_pair(float a, float b, uint32_t &largest) {
  const uint32_t w = pack2<T>(a, b);
  return {T{static_cast<uint16_t>(w)}, T{static_cast<uint16_t>(w >> 16)}};
}
template <>
__device__ __forceinline__ Pair2<float> to_pair<float>(float a, float b, uint32_t &largest) {
  return {a, b};
}
template <>
__device__ __forceinline__ Pair2<Fp16> to_pair<Fp16>(float a, float b, uint32_t &largest) {
  uint32_t w = pack2<Fp16>(a, b);
  asm("{\n\t.reg .b32 m;\n\t"
      "abs.f16x2 m, %0;\n\t"
      "max.f16x2 %1, %1, m;\n\t"
      "min.NaN.f16x2 %0, %0, %2;\n\t"
      "max.NaN.f16x2 %0, %0, %3;\n\t}"
      : "+r"(w), "+r"(largest)
      : "r"(0x7bff7bffu), "r"(0xfbfffbffu));
  return {Fp16{static_cast<uint16_t>(w)}, Fp16{static_cast<uint16_t>(w >> 16)}};
}
__device__ __forceinline__ bool saturated(uint32_t largest) {  // an infinity in either half
  return (largest & 0x7fffu) == 0x7c00u || (largest >> 16 & 0x7fffu) == 0x7c00u;
}

// Arrive on the leader's mbarrier when the accumulator and the ring slot have
// been read.  The arrival and the wait for it have cluster scope, but it
// releases nothing: no memory is handed over (the results are read by later
// launches only), and what may be overwritten afterwards has been read by then
// not by the barrier's order but by completion, of the tensor-memory loads by
// their wait and fence, of the ring slot's by the branch on its values.  A
// release at cluster scope would first wait for the warp's stores of the results
// to reach L2: with it 4096 x 6144 x 1536 takes 85.4k cycles, without 74.1k.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// silu for results of 16 bits from the hardware approximations (relative error
// near 2^-21); with the exact exponential and division for fp32 results.
template <typename T>
__device__ __forceinline__ float silu(float g) {
  return silu_approx(g);
}
template <>
__device__ __forceinline__ float silu<float>(float g) {
  return g * sigmoidf_(g);
}

template <bool kSwiglu, bool kPair, typename T>
__device__ __forceinline__ void gemm_body(const Q8Maps &tmaps, const Q8GemmArgs &p) {
  using C = Cfg<kPair>;
  constexpr int BT = C::BT;
  constexpr uint32_t TMEM_COLS = C::TMEM_COLS;
  constexpr int STAGES = C::STAGES;
  constexpr int A_BYTES = C::A_BYTES;
  constexpr int B_BYTES = C::B_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t *base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t *sA = base;
  uint8_t *sB = base + STAGES * A_BYTES;
  Smem &s = *reinterpret_cast<Smem *>(base + STAGES * C::STAGE_BYTES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int groups = p.groups;
  const int n_tiles = (p.N + C::W_BLOCK - 1) / C::W_BLOCK;
  const int kblocks = (p.K + BK - 1) / BK;
  // token blocks per chunk: about 48 MB of token rows
  const int m_chunk = max(1, (48 << 20) / (BT * p.K));

  // ---- prologue: barriers, tensor memory, per-group tile starts
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], C::EPI_ARRIVALS);
    }
    for (int i = 0; i < TILE_RING; ++i) {
      mbar_init(&s.tile_full[i], 1);
      mbar_init(&s.tile_empty[i], C::EPI_ARRIVALS);
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.draw, 1);
    s.abort_flag = 0;
    s.mma_consumed = 0;
    fence_barrier_init();
    for (int i = 0; i < 3; ++i) tma_prefetch_desc(&tmaps.tok[i]);
    tma_prefetch_desc(&tmaps.w);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&s.tmem_base, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s.tmem_base, TMEM_COLS);
      tmem_relinquish();
    }
  }
  let_next_start();
  previous_done();
  if (threadIdx.x == 64) s.ready = *p.ready == kQ8Ready;
  if (warp == 0) {
    // Group offsets and an exclusive scan of ceil(rows / BT).  The offsets are
    // the caller's: a group whose range is not 0 <= o0 <= o1 <= R, or a first
    // offset other than 0, gets no tiles and is flagged; so is a set of ranges
    // that together hold more rows than there are (the workspace is laid out
    // for max_mtiles token blocks).
    auto offset = [&](int g) { return p.offsets ? p.offsets[g] : (g == 0 ? 0 : p.R); };
    auto token_blocks = [&](int g) {
      const int o0 = offset(g), o1 = offset(g + 1);
      if (o0 < 0 || o1 < o0 || o1 > p.R || (g == 0 && o0 != 0)) {
        record_error(p.err, MOE_ERR_BAD_INDEX);
        return 0;
      }
      return (o1 - o0) / BT + ((o1 - o0) % BT != 0);
    };
    const int per = (groups + 31) / 32;
    const int g0 = lane * per;
    int64_t local = 0;
    for (int g = g0; g < min(g0 + per, groups); ++g) {
      s.grp_off[g] = offset(g);
      local += token_blocks(g);
    }
    int64_t incl = local;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int64_t run = incl - local;
    for (int g = g0; g < min(g0 + per, groups); ++g) {
      s.tile_start[g] = static_cast<int>(run);  // read only if the total fits
      run += token_blocks(g);
    }
    if (lane == 31) {
      s.tile_start[groups] = static_cast<int>(incl);
      if (incl > p.max_mtiles) {
        record_error(p.err, MOE_ERR_BAD_INDEX);
        incl = 0;
      }
      s.total_mtiles = static_cast<int>(incl);
      s.grp_off[groups] = offset(groups);
    }
  }
  tc_fence_before();
  if (kPair)
    cluster_sync();  // the peer's barriers are initialised before any remote use
  else
    __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = s.tmem_base;
  const int total_tiles = s.total_mtiles * n_tiles;
  const bool counted = s.ready != 0;
  const int units = static_cast<int>(gridDim.x) / C::RANKS;
  const int unit = static_cast<int>(blockIdx.x) / C::RANKS;
  // Cut tiles: unit u has part u % parts of tile u / parts.  The number of
  // tiles is only known here, a group's rows being the device's to know.
  const bool cut = p.max_parts > 0 && counted && total_tiles > 0 && total_tiles <= units;
  const int parts = cut ? min(min(p.max_parts, kblocks), units / total_tiles) : 1;
  const int my_tile = unit / parts, my_part = unit - my_tile * parts;
  auto cut_tile = [&](Tile *c) {
    if (my_tile >= total_tiles) return false;
    *c = decode<kPair>(s, p, n_tiles, m_chunk, kblocks, my_tile);
    c->kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * my_part / parts);
    c->kb1 = static_cast<int>(static_cast<int64_t>(kblocks) * (my_part + 1) / parts);
    return true;
  };
  volatile int *abort_flag = &s.abort_flag;
  int issued = 0;  // k-blocks this CTA's producer has loaded

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool elected = elect_one();
    const uint32_t a_smem = smem_addr(sA), b_smem = smem_addr(sB);
    // a pair's loads all complete on the leader's barriers
    const uint32_t full0 = kPair ? cluster_map(&s.full[0], 0) : smem_addr(&s.full[0]);
    uint32_t stage = 0, phase = 0, ts = 0, tph = 0;
    bool ok = true;
    for (bool first = true; ok && !p.stall; first = false) {
      Tile c;
      if (cut) {
        if (!first || !cut_tile(&c)) break;
      } else {
        if (!mbar_wait(&s.tile_full[ts], tph, abort_flag, p.err, kPair)) break;
        const bool any_left = ring_tile(s, ts, kblocks, &c);
        if (++ts == TILE_RING) {
          ts = 0;
          tph ^= 1u;
        }
        if (!any_left) break;
      }
      const int w_row = c.g * p.N + c.w0 + static_cast<int>(rank) * BM;
      const int tok_rows = kPair ? c.n / 2 : c.n;
      const int tok_row0 = c.row_base + static_cast<int>(rank) * tok_rows;
      // one box of 32, 64 or 128 rows holds this CTA's token rows: each TMA
      // instruction costs issue time on the one producing lane
      const int box = tok_rows <= 32 ? 0 : tok_rows <= 64 ? 1 : 2;
      const CUtensorMap *tmap_b = &tmaps.tok[box];
      const uint32_t tx = (kPair ? 2u : 1u) * static_cast<uint32_t>(A_BYTES + (32 << box) * BK);
      const int draw_at = max(c.kb0, c.kb1 - STAGES);
      for (int kb = c.kb0; kb < c.kb1; ++kb) {
        if (leader && !cut && kb == draw_at && lane == 0) mbar_arrive(&s.draw);
        if (!mbar_wait(&s.empty[stage], phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (elected) {
          if (leader) mbar_arrive_expect_tx(&s.full[stage], tx);
          load_tile<kPair>(a_smem + stage * A_BYTES, &tmaps.w, full0 + stage * 8, kb * BK, w_row);
          load_tile<kPair>(b_smem + stage * B_BYTES, tmap_b, full0 + stage * 8, kb * BK, tok_row0);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader) {
      const bool elected = elect_one();
      const uint64_t a_desc0 = umma_desc_sw128(smem_addr(sA)), b_desc0 = umma_desc_sw128(smem_addr(sB));
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, ts = 0, tph = 0;
      int consumed = 0;
      for (bool first = true;; first = false) {
        Tile c;
        if (cut) {
          if (!first || !cut_tile(&c)) break;
        } else {
          if (!mbar_wait(&s.tile_full[ts], tph, abort_flag, p.err)) break;
          const bool any_left = ring_tile(s, ts, kblocks, &c);
          if (++ts == TILE_RING) {
            ts = 0;
            tph ^= 1u;
          }
          if (!any_left) break;
        }
        const uint32_t idesc = idesc_i8(C::W_BLOCK, c.n);
        if (!mbar_wait(&s.tempty[acc], acc_phase ^ 1u, abort_flag, p.err, kPair)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BT;
        bool ok = true;
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          if (!mbar_wait(&s.full[stage], phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          ++consumed;
          if (elected) {
            // a step of 32 bytes of K adds 2 to a descriptor's address field
            const uint64_t a_desc = a_desc0 + stage * (A_BYTES >> 4), b_desc = b_desc0 + stage * (B_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < BK / 32; ++k) {
              const uint32_t accumulate = kb != c.kb0 || k != 0 ? 1u : 0u;
              if (kPair)
                mma_pair(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
              else
                mma(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
            }
            if (kPair)
              umma_commit_pair(&s.empty[stage], 0x3);
            else
              umma_commit(&s.empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elected) {
          if (kPair)
            umma_commit_pair(&s.tfull[acc], 0x3);
          else
            umma_commit(&s.tfull[acc]);
        }
        __syncwarp();
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (lane == 0) s.mma_consumed = consumed;
    }
  } else if (warp == SCHED_WARP) {
    // ------------------------------------------------------------ scheduler (leader)
    // A CTA (or pair) starts on the tile of its own number and draws the
    // following ones from the counter, each when its producer has STAGES
    // k-blocks left to load: late enough that no tile is taken by a CTA that
    // is busy while another is idle, early enough to hide the counter's round
    // trip and the signal to the peer.  (Two ids drawn ahead left 28 of 148
    // CTAs without work, and 24 with two tiles, at 144 tiles.)  In a warp of
    // its own, so that the loads go on meanwhile: drawn by the producer, a
    // tile of 12 k-blocks cost 8.8k cycles instead of 7.7k (20480 tokens on
    // 65 groups of 2048 x 1536: 74.3 -> 69.5 us).
    if (leader && !cut) {
      uint32_t ps = 0, pph = 0, dph = 0;  // next ring slot and its phase, the producer's signal's
      for (int t = unit;;) {
        if (!mbar_wait(&s.tile_empty[ps], pph ^ 1u, abort_flag, p.err, kPair)) break;
        if (lane == 0) {
          // the other roles (and the peer) get the tile's place worked out
          Tile c;
          c.g = -1;
          c.row_base = c.rows = c.w0 = 0;
          if (t < total_tiles) c = decode<kPair>(s, p, n_tiles, m_chunk, kblocks, t);
          *reinterpret_cast<int4 *>(s.tile_ring[ps]) = make_int4(c.g, c.row_base, c.rows, c.w0);
          mbar_arrive(&s.tile_full[ps]);
          if (kPair) {
            const uint32_t peer = cluster_map(s.tile_ring[ps], 1);
            st_shared_remote(peer, c.g);
            st_shared_remote(peer + 4, c.row_base);
            st_shared_remote(peer + 8, c.rows);
            st_shared_remote(peer + 12, c.w0);
            mbar_arrive_remote(cluster_map(&s.tile_full[ps], 1));
          }
        }
        if (t >= total_tiles) break;
        if (++ps == TILE_RING) {
          ps = 0;
          pph ^= 1u;
        }
        if (!mbar_wait(&s.draw, dph, abort_flag, p.err)) break;
        dph ^= 1u;
        // as many draws as tiles: the last one leaves the counter at 0
        if (counted) {
          int drawn = 0;
          if (lane == 0) drawn = static_cast<int>(atomicInc(p.tile_counter, total_tiles - 1));
          t = __shfl_sync(0xffffffffu, drawn, 0) + units;
        } else {
          t += units;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp q = warp % 4 reads tensor-memory lanes 32q .. 32q+31: one weight
    // row (channel) a lane, the tile's token rows along the columns.
    // The warps of a lane quarter take its 32-column chunks in turn.
    const int q = warp & 3;
    constexpr int STEP = EPI_WARPS / 4;
    const int m_first = (warp - 2) / 4;
    uint32_t acc = 0, acc_phase = 0, ts = 0, tph = 0;
    float *row_scale = s.row_scale[warp - 2];
    for (bool first = true;; first = false) {
      Tile c;
      const uint32_t slot = ts;
      if (cut) {
        if (!first || !cut_tile(&c)) break;
      } else {
        if (!mbar_wait(&s.tile_full[ts], tph, abort_flag, p.err, kPair)) break;
        const bool any_left = ring_tile(s, ts, kblocks, &c);
        if (++ts == TILE_RING) {
          ts = 0;
          tph ^= 1u;
        }
        if (!any_left) break;
      }
      const int wr = c.w0 + static_cast<int>(rank) * BM + q * 32;  // this warp's first channel
      const float ws = wr + lane < p.N ? p.w_scale[static_cast<int64_t>(c.g) * p.N + wr + lane] : 0.f;
      // the row scales do not depend on the accumulator: read while the MMAs run
      // (0 for the padding rows, whose results are not stored)
      for (int r = lane; r < c.n; r += 32) row_scale[r] = r < c.rows ? p.x_scale[c.row_base + r] : 0.f;
      __syncwarp();
      // ... and so does the residual: a chunk's 32 rows are read a chunk ahead
      const int ch = wr + lane;
      const bool inside = ch < p.N;
      T res[kSwiglu ? 1 : 32];
      auto load_residual = [&](int m) {
        const int live = min(32, c.rows - 32 * m);
        const T *src = static_cast<const T *>(p.residual) + (c.row_base + 32 * m) * p.ld_residual + ch;
        if (live == 32) {
#pragma unroll
          for (int k = 0; k < 32; ++k, src += p.ld_residual) res[kSwiglu ? 0 : k] = *src;
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k, src += p.ld_residual) {
            if (k >= live) break;
            res[kSwiglu ? 0 : k] = *src;
          }
        }
      };
      const bool any = wr < p.N && 32 * m_first < c.n;  // something to do for this warp
      const bool add = !kSwiglu && p.residual && inside && 32 * m_first < c.rows;
      if (add) load_residual(m_first);
      if (!mbar_wait(&s.tfull[acc], acc_phase, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + acc * BT + (static_cast<uint32_t>(q * 32) << 16);
      bool mine = any;
      // a part's sums: [unit][CTA][column][lane]
      constexpr int64_t SLAB = static_cast<int64_t>(BT) * BM;
      auto slab = [&](int u) {
        return p.partial + (static_cast<int64_t>(u) * C::RANKS + rank) * SLAB + q * 32 + lane;
      };
      const int first_unit = unit - my_part;
      if (parts > 1 && any) {
        int32_t *dst = slab(unit);
        for (int m = m_first; 32 * m < c.n; m += STEP) {
          uint32_t cv[32];
          tmem_ld32(taddr + 32 * m, cv);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) __stcg(dst + (32 * m + k) * BM, static_cast<int32_t>(cv[k]));
        }
        __threadfence();
        __syncwarp();
        int seen = 0;
        if (lane == 0)
          seen = static_cast<int>(
              atomicInc(p.part_counter + (my_tile * C::RANKS + rank) * EPI_WARPS + warp - 2, parts - 1));
        mine = __shfl_sync(0xffffffffu, seen, 0) == parts - 1;
        __threadfence();
      }
      uint32_t largest = 0;
      if (mine) {
        for (int m = m_first; 32 * m < c.n; m += STEP) {
          const int64_t row0 = c.row_base + 32 * m;
          const int live = min(32, c.rows - 32 * m);  // rows of the chunk
          // A store covers one row's 32 channels (SwiGLU: two rows' 16
          // features), so the accumulator needs no transpose.  Full chunks take
          // straight-line code: a test around every store cost more than the
          // MMAs (4096 x 6144 x 2048: 90 us with, 51 without).
          uint32_t cv[32];
          tmem_ld32(taddr + 32 * m, cv);
          tmem_ld_wait();
          for (int u = first_unit; u < first_unit + parts; ++u) {
            if (u == unit) continue;
            const int32_t *src = slab(u) + 32 * m * BM;
#pragma unroll
            for (int k = 0; k < 32; ++k) cv[k] += static_cast<uint32_t>(__ldcg(src + k * BM));
          }
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 xs = *reinterpret_cast<const float4 *>(&row_scale[32 * m + k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k + e] = static_cast<float>(static_cast<int32_t>(cv[k + e]));
            mul2(v[k], v[k + 1], ws, ws);
            mul2(v[k + 2], v[k + 3], ws, ws);
            mul2(v[k], v[k + 1], xs.x, xs.y);
            mul2(v[k + 2], v[k + 3], xs.z, xs.w);
          }
          if (kSwiglu) {
            // lanes 0-15 hold the gate channels of 16 features, lanes 16-31 the
            // up channels: of two rows, the low lanes finish the first and the
            // high lanes the second
            const bool high = lane >= 16;
            T *y = static_cast<T *>(p.y) + (row0 + high) * p.ld_y + wr / 2 + (lane & 15);
            float h[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, high ? v[k] : v[k + 1], 16);
              const float gate = high ? got : v[k], up = high ? v[k + 1] : got;
              h[k / 2] = silu<T>(gate) * up;
            }
            if (live == 32) {
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const Pair2<T> out = to_pair<T>(h[k], h[k + 1], largest);
                *y = out.lo;
                y += 2 * p.ld_y;
                *y = out.hi;
                y += 2 * p.ld_y;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const Pair2<T> out = to_pair<T>(h[k], h[k + 1], largest);
                if (2 * k + high < live) *y = out.lo;
                y += 2 * p.ld_y;
                if (2 * k + 2 + high < live) *y = out.hi;
                y += 2 * p.ld_y;
              }
            }
          } else if (inside) {
            if (add) {
              if (live == 32) {
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] += to_float(res[kSwiglu ? 0 : k]);
              } else {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (k < live) v[k] += to_float(res[kSwiglu ? 0 : k]);
              }
              if (32 * (m + STEP) < c.rows) load_residual(m + STEP);
            }
            T *y = static_cast<T *>(p.y) + row0 * p.ld_y + ch;
            if (live == 32) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const Pair2<T> out = to_pair<T>(v[k], v[k + 1], largest);
                *y = out.lo;
                y += p.ld_y;
                *y = out.hi;
                y += p.ld_y;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                if (k >= live) break;
                const Pair2<T> out = to_pair<T>(v[k], v[k + 1], largest);
                *y = out.lo;
                y += p.ld_y;
                if (k + 1 < live) *y = out.hi;
                y += p.ld_y;
              }
            }
          }
        }
      }
      if (saturated(largest)) record_error(p.err, MOE_ERR_RANGE);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) {
          mbar_arrive(&s.tempty[acc]);
          if (!cut) mbar_arrive(&s.tile_empty[slot]);
        } else {
          arrive_remote(cluster_map(&s.tempty[acc], 0));
          if (!cut) arrive_remote(cluster_map(&s.tile_empty[slot], 0));
        }
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  // ---- teardown.  On the error path wait (bounded) for copies and MMAs still
  // in flight before shared and tensor memory are given back; then both CTAs
  // of the pair meet so neither leaves while the other may still touch its
  // shared memory.
  __syncthreads();
  if (s.abort_flag) {
    if (threadIdx.x == 0) atomicExch(p.ready, 0);
    if (warp == 0 && lane == 0) {
      const uint64_t t0 = global_timer_ns();
      if (leader) {
        for (int i = s.mma_consumed; i < issued; ++i) {
          const uint32_t a = smem_addr(&s.full[i % STAGES]);
          while (!mbar_try_wait(a, static_cast<uint32_t>((i / STAGES) & 1)) &&
                 global_timer_ns() - t0 < kWaitLimitNs) {
          }
        }
      } else {
        while (global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
    // (a commit covers the MMAs of the lane that makes it: the elected one's)
    if (warp == 1 && leader && elect_one()) {
      if (kPair)
        umma_commit_pair(&s.drain, 0x1);
      else
        umma_commit(&s.drain);
      const uint32_t a = smem_addr(&s.drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(a, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else
      tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <bool kSwiglu, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    q8_gemm_pair_kernel(const __grid_constant__ Q8Maps tmaps, Q8GemmArgs p) {
  gemm_body<kSwiglu, true, T>(tmaps, p);
}

template <bool kSwiglu, typename T>
__global__ void __launch_bounds__(THREADS, 1)
    q8_gemm_solo_kernel(const __grid_constant__ Q8Maps tmaps, Q8GemmArgs p) {
  gemm_body<kSwiglu, false, T>(tmaps, p);
}

// As many CTA pairs as can be resident at once (the kernel is persistent), and
// the shared-memory limit raised; asked once per kernel and device.
template <typename Kern>
cudaError_t prepare_kernel(Kern kern, size_t smem, bool pair, int num_sms, int *cached) {
  if (*cached) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  int units = num_sms;
  if (pair) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms & ~1);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&units, kern, &cfg) != cudaSuccess || units <= 0) units = num_sms / 2;
  }
  *cached = units;
  return cudaSuccess;
}

template <bool kSwiglu, typename T>
cudaError_t launch_t(const Q8Maps &tmaps, const Q8GemmArgs &p, bool pair, int num_sms, cudaStream_t stream) {
  static int cached[2][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int &resident = cached[pair ? 1 : 0][dev & 63];
  if (pair) {
    auto kern = q8_gemm_pair_kernel<kSwiglu, T>;
    constexpr size_t smem = smem_bytes<true>();
    e = prepare_kernel(kern, smem, true, num_sms, &resident);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, 2 * static_cast<unsigned>(p.units < resident ? p.units : resident), THREADS, smem,
                             stream, tmaps, p);
  }
  auto kern = q8_gemm_solo_kernel<kSwiglu, T>;
  constexpr size_t smem = smem_bytes<false>();
  e = prepare_kernel(kern, smem, false, num_sms, &resident);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, static_cast<unsigned>(p.units < resident ? p.units : resident), THREADS, smem,
                           stream, tmaps, p);
}
}  // namespace q8

cudaError_t launch_q8_gemm(bool swiglu, int dtype, bool pair, const Q8Maps &tmaps, const Q8GemmArgs &p,
                           int num_sms, cudaStream_t stream) {
  auto go = [&](auto t) {
    using T = decltype(t);
    return swiglu ? q8::launch_t<true, T>(tmaps, p, pair, num_sms, stream)
                  : q8::launch_t<false, T>(tmaps, p, pair, num_sms, stream);
  };
  if (dtype == MOE_DTYPE_BF16) return go(Bf16{});
  if (dtype == MOE_DTYPE_FP16) return go(Fp16{});
  return go(float{});
}

// The tile shape, and how the work is dealt out.
//   CTA pairs or single CTAs: a k-block takes about the same time in either
//   and a pair's covers four times the products per CTA, but a single CTA's
//   tile starts and ends sooner.  Single ones while a group holds at most 64
//   rows (64 x 24576 x 6144: 31.6 us against 33.7; 512 tokens on 64 experts of
//   2048 x 1536: 39.6 against 42.1), and while all their tiles run at once (160 x
//   6144 x 12288: 23.7 against 25.8 us); pairs above (256 x 6144 x 12288: 30.3
//   against 41; 1024 tokens on the 64 experts: 44.9 against 45.1, 1536: 47.0
//   against 54.9).
//   Tiles that are no more than the units are cut into parts where that pays.
//   In k-blocks' time, cutting a tile of kb k-blocks in p parts costs 10 + 4 p
//   for single CTAs and 21 p - 10 for pairs, whose partial sums are four times
//   as large (measured at kb = 16 to 512: 1 x 128 x 65536 whole 92 us, in 4 parts
//   29, in 12 19; 16 x 2048 x 2048 whole 7.3, in 2 parts 8.1; 256 x 6144 x 12288
//   on pairs whole 36.3, in 2 parts 32.0, in 3 33.2).  Shares that straddle tiles,
//   to even out a number of tiles just above the units, cost more than they
//   gave (1 x 24576 x 6144, 192 tiles: 31.8 us against 29.9 dealt out whole).
Q8Plan q8_plan(int64_t R, int N, int K, int groups, int num_sms) {
  Q8Plan p;
  const int64_t touched = R < groups ? R : groups;
  // ceil(rows / bt) summed over groups of R rows in all, at most
  auto blocks = [&](int bt) { return groups == 1 ? (R + bt - 1) / bt : R / bt + touched; };
  p.pair = R > kQ8SoloRows * touched && blocks(kQ8SoloRows) * ((N + 127) / 128) > num_sms;
  const int bt = p.pair ? kQ8PairRows : kQ8SoloRows, wb = p.pair ? 256 : 128;
  const int units = p.pair ? num_sms / 2 : num_sms;
  p.max_mtiles = blocks(bt);
  const int64_t tiles = p.max_mtiles * ((N + wb - 1) / wb);
  p.units = tiles < units ? static_cast<int>(tiles) : units;
  p.max_parts = 0;
  if (tiles > 0 && tiles <= units) {
    const int kb = (K + 127) / 128;
    auto cost = [&](int parts) { return kb / static_cast<double>(parts) + (p.pair ? 21 * parts - 10 : 10 + 4 * parts); };
    p.max_parts = 2;
    while (p.max_parts < kb && cost(p.max_parts + 1) < cost(p.max_parts)) ++p.max_parts;
    if (cost(p.max_parts) >= kb) p.max_parts = 1;
    p.units = static_cast<int>(tiles * (p.max_parts * tiles <= units ? p.max_parts : units / tiles));
  }
  return p;
}

// One part a unit, whatever the other sizes: a workspace for some rows serves
// every product of no more rows.
int64_t q8_partials(int64_t R, int num_sms) {
  return R <= kQ8SoloRows ? int64_t(num_sms) * kQ8SoloRows * 128 : int64_t(num_sms / 2) * 2 * kQ8PairRows * 128;
}

}  // namespace srm
