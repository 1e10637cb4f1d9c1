// kv4_chunk_kernel.cuh - attention over the 4-bit cache for many query rows per cached head
// (include/kv4_b200.h): chunks of prompts, where the tensor cores bound.
//
// The G = Hq / Hkv query heads times N query tokens of one (sequence b, cached head h) are R = G N
// rows over the same keys; a unit is 256 of them, two 128-row tiles that share every converted
// key tile, so a cached value is converted once per 256 rows. On-chip schedule of
// attn_fwd_kernel.cuh (S_t = Q_t K^T and O_t += P_t V on tcgen05 with S, P and O in tensor
// memory, one softmax thread per row, a lazily moved maximum), with these differences:
//  * K^ and V^ do not come by TMA: warps 8-11 read the codes of the next 128-key tile into
//    registers (a thread owns one key row), turn them into f16 (one conversion per two codes and one
//    multiplication by the block scale, both exact) and store them in the 128-byte-swizzled layout
//    that the MMA reads, K^ and V^ double-buffered. Keys behind the sequence's end are stored as
//    zeros. (A deeper ring of raw codes in shared memory instead of registers: 1.13 against 1.05 ms, its copies
//    and loads cost the conversion warps more than the latency they hide.)
//  * q rows are scaled by a power of two and rounded to f16 by their own softmax threads (the
//    bf16 q would need bf16 K^; f16 holds every cached value and gives P three more bits).
//  * The 128-key tiles of all units make one list that is cut into equal runs, one per CTA, as in
//    kv4_attn_kernel.cuh (causal units count only the tiles that their rows see): 148 CTAs of
//    equal work whatever the lengths. A unit that several runs share is joined by
//    kv4_join_sm100 from fp32 parts in the workspace, in the order of the runs.
//  * With at most 128 rows (PAIR) a unit has one row tile, which would leave one softmax group idle and
//    make every step a chain; there both groups work on the same rows, group t on every second key
//    tile, and group 0 joins the two results from tensor memory at the segment's end.
//
// CTA: 16 warps. 0-3 softmax of tile 0, 4-7 of tile 1, 8-11 conversion, 12 MMA issuer (owns
// TMEM), 13 walks the run: it hands out the segments (a unit's tiles [kt0, kt1)) and, tile by
// tile, the cache row of every key through small rings in shared memory, so that neither the page
// lookups nor the walk's state burden the other warps (with every warp walking for itself the
// conversion and softmax warps spilled: 1.50 against 1.05 ms on 2048 queries x 32 heads over 32768
// keys); 14-15 write the rows that see no key. TMEM and MMA order: attn_fwd_kernel.cuh.
// Bound: 4 * 128 * 128 * D operations of a (tile, 128 keys) take 1024 clocks of the tensor pipe at
// D = 128, its 16384 exponentials 1024 clocks of the MUFU units. Measured: 2048 queries x 32 heads (8 cached)
// over 32768 keys, causal: 1.06 ms, 1000 TFLOP/s, 0.60 of the measured bf16 burst rate (0.71 of the sustained; without
// the conversion, which is then wrong, 0.96 ms); a step of two row tiles takes 2.3 us, of which a
// softmax group works 1.5 and waits for its next S the rest. A run starts after 9 us and a further
// segment costs about 6 us: 4 sequences of 238 to 512 queries x 28 heads over 2109 to 4096 keys take 131 to 141 us (470 to
// 510 TFLOP/s).
#pragma once

#include "attn_fwd_kernel.cuh"
#include "kv4_attn_kernel.cuh"

namespace attn {

template <int D_, bool PAIR_>
struct Kv4ChunkCfg {
  static constexpr int D = D_;
  static constexpr bool PAIR = PAIR_;                           // at most 128 rows of a cached head
  static constexpr int CHUNKS = D / 64;                         // 128-byte column chunks of a row of f16
  static constexpr int CHUNK_BYTES = 128 * 128;
  static constexpr int TILE_BYTES = CHUNKS * CHUNK_BYTES;       // 128 rows of f16
  static constexpr int CODE_ROW = D / 2, SF_ROW = D / 16;
  static constexpr int S_KSTEPS = D / 16, PV_KSTEPS = 8;
  static constexpr int P_CHUNKS = 2;                            // (as p_row_to_tmem writes them)
  static constexpr bool PV_F16 = true;
  static constexpr int THREADS = 512;
  static constexpr int CONV_WARP = 8, MMA_WARP = 12, WALK_WARP = 13;
  // launch: 65536 / 512 = 128 registers a thread; 2 * 128 * 184 + 128 * 96 + 128 * 48 = 65536
  static constexpr uint32_t REGS_SOFTMAX = 184, REGS_CONV = 96, REGS_MMA = 48;
  static_assert(2 * REGS_SOFTMAX + REGS_CONV + REGS_MMA <= 512, "register split");
  static constexpr uint32_t TMEM_COLS = 512, O_COL0 = 256;
  static constexpr int SMEM_Q = 0;                              // 2 tiles
  static constexpr int SMEM_K = 2 * TILE_BYTES;                 // 2 buffers
  static constexpr int SMEM_V = 4 * TILE_BYTES;                 // 2 buffers
  static constexpr int SMEM_BAR = 6 * TILE_BYTES;
  static constexpr int RING = 4;                                // segments, and tiles, handed out ahead
  // q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2][2], o_done[2], drain,
  // seg_full[RING], seg_empty[RING], row_full[RING], row_empty[RING], xch_full, xch_empty
  static constexpr int NUM_BARS = 2 * 7 + 4 + 1 + 4 * RING + 2;
  static constexpr int SMEM_MISC = SMEM_BAR + (NUM_BARS + 1) / 2 * 16;
  static constexpr int SMEM_SEG = SMEM_MISC + 16;               // Kv4Seg[RING]
  static constexpr int SMEM_ROWS = SMEM_SEG + RING * 64;        // [RING][128] cache rows, [RING] whether there is a tile
  static constexpr int SMEM_XCH = SMEM_ROWS + RING * (128 + 4) * 4;       // PAIR: [128] (max, sum) of group 1
  static constexpr int SMEM_STAGE = SMEM_XCH + 128 * 8;         // output rows: 2 KB per softmax warp
  static constexpr int SMEM_BYTES = SMEM_STAGE + 8 * 2048 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};
constexpr int kChunkRows = 256;

// A segment as the walking warp hands it out.
struct __align__(16) Kv4Seg {
  int kt0, kt1;              // its key tiles (kt0 == kt1: the run is over)
  int end[2];                // the row tiles see keys up to these tiles (at most kt1)
  int len, n;                // of the sequence
  int r0, slot;              // first row of the unit in (b, h); part slot, or -1 for a whole unit
  unsigned long long row;    // row of (b, h, 0) in q and o
};
static_assert(sizeof(Kv4Seg) <= 64, "segment ring");
template <int D>
struct SfWords { static constexpr int N = D / 64; };   // 32-bit words of a row's scale bytes

struct Kv4ChunkParams {
  Kv4AttnParams a;           // part_o: [2 ctas][256][D], part_ml: [2 ctas][256]; row_blocks = ceil(R / 256)
  uint64_t timeout_cycles;   // per pipeline wait, in SM cycles
  int fault_cta;             // testing only: this CTA's walk withholds its first key tile (-1: none)
};

// Key tiles that the 128 rows from r0 of sequence (len, n) see.
__device__ __forceinline__ int kv4_row_tiles(const Kv4AttnParams& p, int len, int n, int r0, int R) {
  if (r0 >= R || n == 0) return 0;
  const int span = min(128, R - r0), i0 = r0 % p.N;
  const bool wraps = i0 + span > p.N;                // the rows reach into the next head
  if (i0 >= n && !wraps) return 0;
  if (!p.causal) return (len + 127) >> 7;
  const int most = i0 < n ? (wraps ? n - 1 : min(n - 1, i0 + span - 1)) : min(n - 1, i0 + span - p.N - 1);
  return (max(0, min(len, len - n + most + 1)) + 127) >> 7;
}

// The cut of `units` tiles into runs: CTA c of n = min(ctas, units) takes [start(c), start(c + 1)). (Units that count
// for more than their tiles, as items do in Kv4Runs, gained nothing here: four uneven chunks of up to 512 tokens after
// up to 4096 keys, 28 query heads on 4, 135 to 140 us either way.)
struct Kv4ChunkRuns {
  long long units;
  int n;
  __device__ __forceinline__ Kv4ChunkRuns(long long u, int ctas) : units(u), n(static_cast<int>(u < ctas ? u : ctas)) {}
  __device__ __forceinline__ long long start(int c) const { return units * c / n; }
  __device__ __forceinline__ int cta_of(long long u) const { return static_cast<int>(((u + 1) * n - 1) / units); }
};

// Walks a run's segments: tiles [kt0, kt1) of unit (b, qp, h), its two row tiles seeing keys up to
// tile end[t]. Units are ordered by sequence, row pair, head.
struct Kv4ChunkWalk {
  const Kv4AttnParams& p;
  int R;
  long long u, u_end, first;                         // first: first tile of (b, qp)
  long long mine0;                                   // tiles of the lane's (b, qp) entries, from total()
  int b, qp, h, len, n, kt0, kt1, nkv;
  int end[2];

  __device__ __forceinline__ explicit Kv4ChunkWalk(const Kv4AttnParams& params)
      : p(params), R(params.Hq / params.c.H * params.N) {}

  // tiles of one head of (b, qp) = idx
  __device__ __forceinline__ int tiles(int idx) {
    const int bb = idx / p.row_blocks, q = idx - bb * p.row_blocks;
    const int l = kv4_len(p.c, bb), nn = kv4_qlen(p, bb);
    return max(kv4_row_tiles(p, l, nn, q * kChunkRows, R), kv4_row_tiles(p, l, nn, q * kChunkRows + 128, R));
  }
  // total tiles (the whole warp takes part)
  __device__ __forceinline__ long long total(int lane) {
    long long s = 0;
    for (int i = lane; i < p.c.B * p.row_blocks; i += 32) s += tiles(i);
    mine0 = s * p.c.H;
#pragma unroll
    for (int t = 16; t > 0; t >>= 1) s += __shfl_xor_sync(0xffffffffu, s, t);
    return s * p.c.H;
  }
  // to the run [u0, u1) (the whole warp takes part)
  __device__ __forceinline__ void seek(long long u0, long long u1, int lane) {
    u = u0;
    u_end = u1;
    first = 0;
    for (int i0 = 0;; i0 += 32) {
      const long long mine = p.c.B * p.row_blocks <= 32 ? mine0
                             : i0 + lane < p.c.B * p.row_blocks ? static_cast<long long>(tiles(i0 + lane)) * p.c.H : 0;
      long long incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, first + incl > u);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        b = (i0 + l) / p.row_blocks;
        qp = (i0 + l) % p.row_blocks;
        first += __shfl_sync(0xffffffffu, incl - mine, l);
        break;
      }
      first += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // the segment that starts at u (u < u_end); moves u behind it
  __device__ __forceinline__ void next() {
    for (;;) {
      len = kv4_len(p.c, b);
      n = kv4_qlen(p, b);
      end[0] = kv4_row_tiles(p, len, n, qp * kChunkRows, R);
      end[1] = kv4_row_tiles(p, len, n, qp * kChunkRows + 128, R);
      nkv = max(end[0], end[1]);
      if (u < first + static_cast<long long>(nkv) * p.c.H) break;
      first += static_cast<long long>(nkv) * p.c.H;
      if (++qp == p.row_blocks) qp = 0, ++b;
    }
    const uint32_t off = static_cast<uint32_t>(u - first);
    h = static_cast<int>(off / static_cast<uint32_t>(nkv));
    kt0 = static_cast<int>(off - static_cast<uint32_t>(h) * nkv);
    kt1 = static_cast<int>(min(static_cast<long long>(nkv), kt0 + (u_end - u)));
    u += kt1 - kt0;
    end[0] = min(end[0], kt1);
    end[1] = min(end[1], kt1);
  }
  __device__ __forceinline__ bool whole() const { return kt0 == 0 && kt1 == nkv; }
};

template <class C, bool F16>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_chunk_sm100(const Kv4ChunkParams cp) {
  using namespace b200;
  constexpr int D = C::D;
  const Kv4AttnParams& p = cp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::SMEM_BAR);
  uint64_t* k_full = q_full + 2;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;
  uint64_t* p_full = s_full + 2;                     // [tile][chunk]
  uint64_t* o_done = p_full + 4;
  uint64_t* drain_bar = o_done + 2;
  uint64_t* seg_full = drain_bar + 1;
  uint64_t* seg_empty = seg_full + C::RING;
  uint64_t* row_full = seg_empty + C::RING;
  uint64_t* row_empty = row_full + C::RING;
  uint64_t* xch_full = row_empty + C::RING;          // PAIR: group 1's result is complete
  uint64_t* xch_empty = xch_full + 1;                // and has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC);
  uint32_t* abort_word = tmem_slot + 1;
  volatile uint32_t* zeroed = tmem_slot + 2;         // a NaN value was stored as zero (see the conversion)
  Kv4Seg* segs = reinterpret_cast<Kv4Seg*>(smem + C::SMEM_SEG);
  static_assert(sizeof(Kv4Seg) * C::RING <= C::SMEM_ROWS - C::SMEM_SEG, "segment ring");
  uint32_t* rows = reinterpret_cast<uint32_t*>(smem + C::SMEM_ROWS);      // [RING][128]
  uint32_t* is_tile = rows + C::RING * 128;          // [RING]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  kv4_grid_wait();
  asm volatile("griddepcontrol.launch_dependents;");

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + 2 * i, 128);
      mbar_init(p_full + 2 * i + 1, 128);
      mbar_init(o_done + i, 1);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(seg_full + i, 1);
      mbar_init(seg_empty + i, 9);                   // eight softmax warps, the MMA warp
      mbar_init(row_full + i, 1);
      mbar_init(row_empty + i, 4);                   // conversion warps
    }
    mbar_init(xch_full, 128);
    mbar_init(xch_empty, 128);
    *abort_word = 0u;
    *zeroed = 0u;
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Waiter waiter{abort_word, cp.timeout_cycles};
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, waiter.wait(bar, parity)); };
  bool ok = true;
  // segment number sg of the run: waits for it, and gives it back
  auto take_segment = [&](uint32_t sg) { return wait_all(seg_full + sg % C::RING, (sg / C::RING) & 1u); };
  auto free_segment = [&](uint32_t sg) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + sg % C::RING);
  };

  if (warp >= C::MMA_WARP) {
    // ======================= MMA issuer =======================
    regs_decrease<C::REGS_MMA>();
    if (warp == C::MMA_WARP) {
      const uint32_t leader = elect_one() ? 1u : 0u;
      auto commit = [&](uint64_t* bar) { mma_commit(bar, leader); };
      constexpr uint32_t idesc_s = instr_desc(0u, 128, 128, 0, 0);
      constexpr uint32_t idesc_o = instr_desc(0u, 128, D, 0, 1);
      constexpr uint32_t hi = smem_desc_hi(1024);
      const uint32_t q_lo = smem_desc_lo(smem_addr(smem + C::SMEM_Q), 16);
      const uint32_t k_lo = smem_desc_lo(smem_addr(smem + C::SMEM_K), 16);
      const uint32_t v_lo = smem_desc_lo(smem_addr(smem + C::SMEM_V), C::CHUNK_BYTES);
      auto issue_s = [&](int t, uint32_t buf) {      // S_t; PAIR: of the one q tile
        const uint32_t qa = q_lo + (((C::PAIR ? 0 : t) * C::TILE_BYTES) >> 4), ka = k_lo + ((buf * C::TILE_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < C::S_KSTEPS; ++kk) {
          const uint32_t off = ((kk / 4) * C::CHUNK_BYTES + (kk % 4) * 32) >> 4;
          mma_f16_ss(tmem_base + t * 128, smem_desc(qa + off, hi), smem_desc(ka + off, hi), idesc_s, kk > 0, leader);
        }
      };
      auto issue_pv = [&](int t, uint32_t buf, int c, bool acc) {
        const uint32_t va = v_lo + ((buf * C::TILE_BYTES) >> 4);
#pragma unroll
        for (int i = 0; i < C::PV_KSTEPS / 2; ++i) {
          const int kv = c * (C::PV_KSTEPS / 2) + i;
          mma_f16_ts(tmem_base + C::O_COL0 + t * D, tmem_base + t * 128 + kv * 8, smem_desc(va + ((kv * 16 * 128) >> 4), hi),
                     idesc_o, (acc || i > 0) ? 1u : 0u, leader);
        }
      };
      uint32_t k = 0;                                // key tiles used so far
      uint32_t qc = 0, pc = 0;                       // phases of q_full and p_full: bit t
      for (uint32_t sg = 0; (ok = take_segment(sg)); ++sg) {
        const Kv4Seg& from = segs[sg % C::RING];
        struct {
          int kt0, kt1, end[2];
        } const w{from.kt0, from.kt1, {from.end[0], from.end[1]}};
        free_segment(sg);
        if (w.kt0 == w.kt1) break;
        if constexpr (C::PAIR) {
          // group t takes the segment's key tiles t, t + 2, ...: S of the first two, then for each tile
          // its P V and the S of the next but one
          auto s_of = [&](int t, uint32_t x) -> bool {     // S_t of the run's key tile x
            if (!wait_all(k_full + (x & 1), (x >> 1) & 1)) return false;
            tc_fence_after();
            issue_s(t, x & 1);
            commit(s_full + t);
            commit(k_empty + (x & 1));
            return true;
          };
          const int nt = w.kt1 - w.kt0;
          if (!(ok = wait_all(q_full, qc & 1u))) break;
          qc ^= 1u;
          if (!(ok = s_of(0, k)) || (nt > 1 && !(ok = s_of(1, k + 1)))) break;
          for (int j = 0; j < nt; ++j, ++k) {
            const int t = j & 1;
            if (!(ok = wait_all(v_full + (k & 1), (k >> 1) & 1))) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (!(ok = wait_all(p_full + 2 * t + c, (pc >> t) & 1u))) break;
              tc_fence_after();
              issue_pv(t, k & 1, c, j > 1 || c > 0);
            }
            if (!ok) break;
            pc ^= 1u << t;
            if (j + 2 >= nt) commit(o_done + t);
            commit(v_empty + (k & 1));
            if (j + 2 < nt && !(ok = s_of(t, k + 2))) break;
          }
          if (!ok) break;
        } else {
          // S of the segment's first tile (issued after the previous segment's last P V on this
          // thread, so it overwrites that P only after it has been read)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (w.end[t] > w.kt0) {
              if (!(ok = wait_all(q_full + t, (qc >> t) & 1u))) break;
              qc ^= 1u << t;
            }
          if (!ok || !(ok = wait_all(k_full + (k & 1), (k >> 1) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (w.end[t] > w.kt0) {
              issue_s(t, k & 1);
              commit(s_full + t);
            }
          commit(k_empty + (k & 1));
          for (int j = w.kt0; j < w.kt1; ++j, ++k) {
            const uint32_t k1 = k + 1;
            if (!(ok = wait_all(v_full + (k & 1), (k >> 1) & 1))) break;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (j >= w.end[t]) continue;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (!(ok = wait_all(p_full + 2 * t + c, (pc >> t) & 1u))) break;
                tc_fence_after();
                issue_pv(t, k & 1, c, j > w.kt0 || c > 0);
              }
              if (!ok) break;
              pc ^= 1u << t;
              if (j + 1 < w.end[t]) {
                if (!k_ready) {
                  if (!(ok = wait_all(k_full + (k1 & 1), (k1 >> 1) & 1))) break;
                  k_ready = true;
                  tc_fence_after();
                }
                issue_s(t, k1 & 1);
                commit(s_full + t);
              } else {
                commit(o_done + t);
              }
            }
            if (!ok) break;
            commit(v_empty + (k & 1));
            if (k_ready) commit(k_empty + (k1 & 1));
          }
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) record_timeout();
      // every MMA this warp issued completes before TMEM can be released
      commit(drain_bar);
      drain_wait(drain_bar, 0, cp.timeout_cycles);
      __syncwarp();
    } else if (warp == C::WALK_WARP) {
      // ======================= the walk =======================
      Kv4ChunkWalk w(p);
      const Kv4ChunkRuns runs(w.total(lane), p.ctas);
      const bool idle = static_cast<int>(blockIdx.x) >= runs.n;
      const long long u0 = idle ? 0 : runs.start(blockIdx.x), u1 = idle ? 0 : runs.start(blockIdx.x + 1);
      if (!idle) w.seek(u0, u1, lane);
      w.u = u0;
      w.u_end = u1;
      if (lane == 0) p.heads[blockIdx.x].parts = 0;
      const uint32_t slot_mask = (1u << p.c.page_shift) - 1u;
      uint32_t k = 0;
      for (uint32_t sg = 0; ok; ++sg) {
        const bool over = w.u >= w.u_end, first = w.u == u0;
        if (!over) w.next();
        if (sg >= C::RING && !(ok = wait_all(seg_empty + sg % C::RING, (sg / C::RING - 1) & 1u))) break;
        if (lane == 0) {
          Kv4Seg x;
          x.kt0 = over ? 0 : w.kt0, x.kt1 = over ? 0 : w.kt1;
          x.end[0] = over ? 0 : w.end[0], x.end[1] = over ? 0 : w.end[1];
          x.len = w.len, x.n = w.n;
          x.r0 = w.qp * kChunkRows;
          x.slot = !over && w.whole() ? -1 : 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1);
          x.row = (static_cast<unsigned long long>(w.b) * p.c.H + w.h) * w.R;
          segs[sg % C::RING] = x;
          if (!over && w.kt0 == 0 && !w.whole()) {    // the unit's first part: what the join needs
            Kv4Head hd;
            hd.parts = runs.cta_of(w.u - w.kt1 + w.nkv - 1) - static_cast<int>(blockIdx.x) + 1;
            hd.b = w.b, hd.h = w.h, hd.rb = w.qp, hd.slot = x.slot;
            p.heads[blockIdx.x] = hd;
          }
          mbar_arrive(seg_full + sg % C::RING);
        }
        if (over) break;
        const int* table = p.c.block_table + static_cast<long long>(w.b) * p.c.max_pages;
        for (int j = w.kt0; j < w.kt1; ++j, ++k) {
          uint32_t rw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = j * 128 + 32 * i + lane;
            rw[i] = key < w.len ? static_cast<uint32_t>(table[key >> p.c.page_shift]) : kNoRow;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = j * 128 + 32 * i + lane;
            uint32_t row;
            rw[i] = key < w.len && kv4_row(p.c, static_cast<int>(rw[i]), w.h, key & static_cast<int>(slot_mask), row)
                        ? row : kNoRow;
          }
          const uint32_t at = k % C::RING;
          if (k >= C::RING && !(ok = wait_all(row_empty + at, (k / C::RING - 1) & 1u))) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) rows[at * 128 + 32 * i + lane] = rw[i];
          if (lane == 0) is_tile[at] = 1u;
          __syncwarp();
          // (testing hook: a tile that is never handed out; the bounded waits on it run out)
          if (lane == 0 && !(k == 0 && static_cast<int>(blockIdx.x) == cp.fault_cta)) mbar_arrive(row_full + at);
        }
      }
      // the conversion warps stop at the tile that says so
      if (ok) {
        const uint32_t at = k % C::RING;
        if (k >= C::RING) ok = wait_all(row_empty + at, (k / C::RING - 1) & 1u);
        if (lane == 0) {
          is_tile[at] = 0u;
          mbar_arrive(row_full + at);
        }
      }
      if (!ok && lane == 0) record_timeout();
      __syncwarp();
    } else {
      kv4_empty_rows<D>(p, threadIdx.x - (C::WALK_WARP + 1) * 32, 64);
    }
  } else if (warp >= C::CONV_WARP) {
    // ======================= codes -> f16 K^ and V^ =======================
    regs_decrease<C::REGS_CONV>();
    const int kr = threadIdx.x - C::CONV_WARP * 32;   // key row of this thread
    constexpr int NW = C::CODE_ROW / 16;              // 16-byte pieces of a row's codes
    uint4 kw[NW], vw[NW];
    uint32_t ksf[SfWords<D>::N], vsf_next[SfWords<D>::N], vsf[SfWords<D>::N];
    uint32_t row = kNoRow;                            // cache row of this thread's key in the tile loaded last
    // tile k of the run: its row, K's codes and the scales of both; false: there is none
    auto load_k = [&](uint32_t k) {
      const uint32_t at = k % C::RING;
      if (!(ok = wait_all(row_full + at, (k / C::RING) & 1u))) return false;
      const bool found = is_tile[at] != 0u;
      row = rows[at * 128 + kr];
      __syncwarp();
      if (lane == 0) mbar_arrive(row_empty + at);
      if (!found) return false;
#pragma unroll
      for (int i = 0; i < SfWords<D>::N; ++i) ksf[i] = vsf_next[i] = 0u;
#pragma unroll
      for (int i = 0; i < NW; ++i) kw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row != kNoRow) {
        const uint4* src = reinterpret_cast<const uint4*>(p.c.codes[0] + static_cast<size_t>(row) * C::CODE_ROW);
#pragma unroll
        for (int i = 0; i < NW; ++i) kw[i] = src[i];
#pragma unroll
        for (int i = 0; i < SfWords<D>::N; ++i) {
          ksf[i] = reinterpret_cast<const uint32_t*>(p.c.sf[0] + static_cast<size_t>(row) * C::SF_ROW)[i];
          vsf_next[i] = reinterpret_cast<const uint32_t*>(p.c.sf[1] + static_cast<size_t>(row) * C::SF_ROW)[i];
        }
      }
      return true;
    };
    auto load_v = [&]() {
#pragma unroll
      for (int i = 0; i < NW; ++i) vw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row != kNoRow) {
        const uint4* src = reinterpret_cast<const uint4*>(p.c.codes[1] + static_cast<size_t>(row) * C::CODE_ROW);
#pragma unroll
        for (int i = 0; i < NW; ++i) vw[i] = src[i];
      }
    };
    // a row of D f16 values, written to row kr of the tile at dst
    auto convert = [&](const uint4 (&cw)[NW], const uint32_t (&sf)[SfWords<D>::N], uint8_t* dst) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {                  // 32 values, two blocks
        const uint32_t s2 = f16x2_from_e4m3x2(static_cast<uint16_t>(sf[i >> 1] >> (16 * (i & 1))));
        const uint32_t wds[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {                 // 8 values: one 16-byte unit of the f16 row
          uint32_t f[4];
          f16x2_from_e2m1x8(wds[q], f);
          const uint32_t sc = q < 2 ? splat_lo(s2) : splat_hi(s2);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = hmul2(f[e], sc);
          const int un = 4 * i + q;
          *reinterpret_cast<uint4*>(dst + (un >> 3) * C::CHUNK_BYTES + kr * 128 + (((un & 7) ^ (kr & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
    };
    bool more = load_k(0);
    if (more) load_v();
    for (uint32_t k = 0; more; ++k) {
      const uint32_t buf = k & 1u, round = k >> 1;
#pragma unroll
      for (int i = 0; i < SfWords<D>::N; ++i) vsf[i] = vsf_next[i];
      // A NaN value must reach the rows that see it and no other, and P = 0 would not keep it from a
      // masked row: NaN blocks of values are stored as zeros, and the rows that see them get their NaN
      // where the segment is written (`zeroed` says that this has happened in the run; the mark is set before
      // k_full, and so before that segment's last P V).
#pragma unroll
      for (int i = 0; i < SfWords<D>::N; ++i) {
        const uint32_t nan = nan_scales(vsf[i]);
        if (nan != 0u) {
          vsf[i] &= ~nan;
          *zeroed = 1u;
        }
      }
      if (k >= 2 && !(ok = wait_all(k_empty + buf, (round - 1) & 1))) break;
      convert(kw, ksf, smem + C::SMEM_K + buf * C::TILE_BYTES);
      fence_proxy_async_shared();   // the MMA (async proxy) reads what these threads wrote
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + buf);
      more = load_k(k + 1);
      if (!ok) break;
      if (k >= 2 && !(ok = wait_all(v_empty + buf, (round - 1) & 1))) break;
      convert(vw, vsf, smem + C::SMEM_V + buf * C::TILE_BYTES);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + buf);
      if (more) load_v();
    }
    if (!ok && lane == 0) record_timeout();
  } else {
    // ======================= softmax: one thread per row =======================
    regs_increase<C::REGS_SOFTMAX>();
    const int t = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_tm = tmem_base + lane_off + t * 128;
    const uint32_t o_tm = tmem_base + lane_off + C::O_COL0 + t * D;
    uint32_t sc = 0, oc = 0;                          // phases of s_full and o_done
    const int R = p.Hq / p.c.H * p.N;
    // A row of q or of 16-bit output is UPR 16-byte units; RPI rows make 32 of them.
    constexpr int UPR = D / 8, RPI = 32 / UPR;
    // (the thread's place is read anew, opaquely, where a segment begins and ends: what is derived from it
    // would otherwise be kept in registers through the tile loop, which spills for it)
    auto thread_here = [] {
      uint32_t x;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
      return static_cast<int>(x);
    };
    // Copies the q rows of segment sg to the warp's rows of this group's q tile, whole rows to consecutive
    // lanes (zeros behind the last row). The tile is free: every S MMA that read it has completed when
    // this group has seen its last S. PAIR: group 1 fills the second tile's place with the same rows for
    // itself; the MMA reads group 0's.
    auto copy_q = [&](uint32_t sg) {
      volatile const Kv4Seg& w = segs[sg % C::RING];
      const int here = thread_here(), ln = here & 31, w0 = (here & 127) & ~31, tile = here >> 7;
      if (C::PAIR ? w.kt0 + tile < w.kt1 : w.kt0 < w.end[tile]) {
        const int row0 = w.r0 + (C::PAIR ? 0 : tile * 128) + w0;
        const uint8_t* src = p.q + (w.row + row0) * (D * 2) + (ln % UPR) * 16;
        const uint32_t dst = smem_addr(smem + C::SMEM_Q + tile * C::TILE_BYTES) + ((ln % UPR) >> 3) * C::CHUNK_BYTES;
#pragma unroll 1   // (unrolled, ptxas schedules the tile loop worse: 1.12 against 1.04 ms)
        for (int it = 0; it < UPR; ++it) {
          const int i = it * RPI + ln / UPR, rw = w0 + i;
          const bool valid = row0 + i < R;
          cp_async_16z(dst + rw * 128 + ((((ln % UPR) & 7) ^ (rw & 7)) << 4), valid ? src + static_cast<size_t>(i) * D * 2 : p.q,
                       valid);
        }
      }
      cp_async_commit();
    };
    uint32_t xc = 0;                                  // PAIR: segments so far (phases of xch_full, xch_empty)
    float2* xch = reinterpret_cast<float2*>(smem + C::SMEM_XCH);
    if ((ok = take_segment(0))) copy_q(0);
    for (uint32_t sg = 0; ok; ++sg) {
      // (read again after the tile loop, which has no registers to spare for the segment's fields)
      volatile const Kv4Seg& w = segs[sg % C::RING];
      const int j0 = w.kt0 + (C::PAIR ? t : 0), endt = C::PAIR ? w.kt1 : w.end[t];   // this group's key tiles:
      constexpr int STEP = C::PAIR ? 2 : 1;                                            // j0, j0 + STEP, ... < endt
      if (w.kt0 == w.kt1) break;
      int lim;                                        // last key this row sees
      {
        const int here = thread_here(), tile_row = C::PAIR ? here & 127 : here & 255;
        const int i_tok = (w.r0 + tile_row) % p.N;    // (rows that hold no query see everything: they are not written)
        lim = p.causal && i_tok < w.n ? w.len - w.n + i_tok : w.len - 1;
        if (!C::PAIR && endt <= j0) {
          if (w.slot >= 0) p.part_ml[static_cast<size_t>(w.slot) * kChunkRows + tile_row] = make_float2(-INFINITY, 0.f);
          free_segment(sg);
          if ((ok = take_segment(sg + 1))) copy_q(sg + 1);
          continue;
        }
      }
      // ---- q has been copied (see copy_q); each row is scaled by a power of two and becomes f16 in
      // place, a thread per row. PAIR: group 0 does it for both, group 1 only needs the factor.
      float c = 1.f;
      if (j0 < endt) {
        cp_async_wait<0>();
        __syncwarp();
        const int here = thread_here(), row = here & 127;
        uint8_t* const tile_rows = smem + C::SMEM_Q + (here >> 7) * C::TILE_BYTES;
        auto unit = [&](int u) {
          return reinterpret_cast<uint4*>(tile_rows + (u >> 3) * C::CHUNK_BYTES + row * 128 + (((u & 7) ^ (row & 7)) << 4));
        };
        float amax = 0.f;
#pragma unroll 4
        for (int u = 0; u < D / 8; ++u) {
          const uint4 x = *unit(u);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = f32x2_from_16<F16>(xs[e]);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        const int e2 = kv4_row_exp(amax);
        c = fmaxf(__int_as_float(e2 << 23) * p.scale_log2, 1e-37f);
        if (!C::PAIR || t == 0) {
          const float down = __int_as_float((254 - e2) << 23);
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) {
            const uint4 x = *unit(u);
            uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = f32x2_from_16<F16>(xs[e]);
              xs[e] = pack_f16x2(f.x * down, f.y * down);
            }
            *unit(u) = make_uint4(xs[0], xs[1], xs[2], xs[3]);
          }
          fence_proxy_async_shared();
          mbar_arrive(q_full + (C::PAIR ? 0 : t));
        }
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = j0; j < endt; j += STEP) {
        if (!(ok = wait_all(s_full + t, sc & 1))) break;
        ++sc;
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(s_tm + 0, sr + 0);
        tmem_ld32(s_tm + 32, sr + 32);
        tmem_ld32(s_tm + 64, sr + 64);
        tmem_ld32(s_tm + 96, sr + 96);
        tmem_ld_wait<128>(sr);
        const int limit = lim - j * 128;
        if (__any_sync(0xffffffffu, limit < 127)) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > limit) sr[i] = 0xff800000u;       // -inf
        }
        const float m_blk = row_max128(sr) * c;
        float m_use = m_run;
        if (kv4_outgrown(m_blk, m_run)) m_use = kv4_below(m_blk);
        const bool moved = m_use != m_run;
        const float alpha = moved ? ex2_approx(m_run - m_use) : 1.f;
        if (j > j0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int cb = 0; cb < D; cb += 32) {
            uint32_t ov[32];
            tmem_ld32(o_tm + cb, ov);
            tmem_ld_wait<32>(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(o_tm + cb, ov);
          }
        }
        // (a row that has seen no key yet: every score is -infinity, every P 0)
        const float sum = p_row_to_tmem<C, 0u>(sr, c, m_use == -INFINITY ? 0.f : m_use, s_tm, p_full + 2 * t);
        l_run = l_run * alpha + sum;
        m_run = m_use;
      }
      if (!ok) break;
      // the next segment's q comes in under this one's last P V and its output (PAIR: group 1's S MMAs
      // read group 0's tile too, so that group 0 copies once group 1's result is complete)
      if (!(ok = take_segment(sg + 1))) break;
      if (!C::PAIR || t == 1) copy_q(sg + 1);
      if (!C::PAIR || j0 < endt) {
        if (!(ok = wait_all(o_done + t, oc & 1))) break;
        ++oc;
        tc_fence_after();
      }
      const int here = thread_here(), lane = here & 31, wq = (here >> 5) & 3, ta = C::PAIR ? 0 : here >> 7;
      const int r = wq * 32 + lane;
      // output rows pass through shared memory, 64 bytes of each of the warp's 32 at a time, so that
      // consecutive lanes write whole sectors of a row
      uint8_t* const stage = smem + C::SMEM_STAGE + (here >> 5) * 2048;
      auto unit_at = [&](int i, int u) { return reinterpret_cast<uint4*>(stage + i * 64 + ((u ^ ((i >> 1) & 3)) << 4)); };
      const bool whole = w.slot < 0;
      const int row0 = w.r0 + ta * 128 + wq * 32;
      const unsigned long long qrow0 = w.row + row0;
      const bool write = row0 + lane < R && (row0 + lane) % p.N < w.n;
      const size_t prow = static_cast<size_t>(whole ? 0 : w.slot) * kChunkRows + ta * 128 + r;
      float f0 = 1.f, f1 = 0.f;                       // factors of this group's O and of group 1's
      if constexpr (C::PAIR) {
        const uint32_t ph = xc & 1u;
        ++xc;
        if (t == 1) {                                 // hands its result over, and waits until it has been read
          xch[r] = make_float2(m_run, l_run);
          tc_fence_before();
          mbar_arrive(xch_full);
          if (!(ok = wait_all(xch_empty, ph))) break;
          tc_fence_after();
          free_segment(sg);
          continue;
        }
        if (!(ok = wait_all(xch_full, ph))) break;
        tc_fence_after();
        copy_q(sg + 1);
        const float2 x = xch[r];
        const float M = fmaxf(m_run, x.x), Mu = M == -INFINITY ? 0.f : M;
        f0 = ex2_approx(m_run - Mu);
        f1 = ex2_approx(x.x - Mu);
        l_run = l_run * f0 + x.y * f1;
        m_run = M;
      }
      if (whole) {
        const float inv = kv4_norm(p, l_run, lim >= 0);
        f0 *= inv;
        f1 *= inv;
      }
      const bool join = C::PAIR && w.kt1 - w.kt0 > 1; // group 1 had a tile
      const uint32_t wmask = __ballot_sync(0xffffffffu, write);
      uint8_t* const gout = whole ? p.o + qrow0 * D * 2
                                  : reinterpret_cast<uint8_t*>(p.part_o + (prow - lane) * static_cast<size_t>(D));
      // the staged 64 bytes of every row to bytes [at, at + 64) of its row of `bytes` bytes
      auto flush = [&](int bytes, int at) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int i = it * 8 + lane / 4;
          const uint4 x = *unit_at(i, lane & 3);
          if (!whole || ((wmask >> i) & 1u))
            *reinterpret_cast<uint4*>(gout + static_cast<size_t>(i) * bytes + at + (lane & 3) * 16) = x;
        }
        __syncwarp();
      };
#pragma unroll
      for (int cb = 0; cb < D; cb += 32) {
        uint32_t ov[32];
        tmem_ld32(o_tm + cb, ov);
        tmem_ld_wait<32>(ov);
        if (C::PAIR || whole) {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f0);
        }
        if (join) {
          uint32_t o1[32];
          tmem_ld32(o_tm + D + cb, o1);
          tmem_ld_wait<32>(o1);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ov[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(ov[i])));
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pk[e] = pack_16<F16>(__uint_as_float(ov[8 * i + 2 * e]), __uint_as_float(ov[8 * i + 2 * e + 1]));
            *unit_at(lane, i) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          flush(D * 2, cb * 2);
        } else {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *unit_at(lane, i) = make_uint4(ov[16 * hf + 4 * i], ov[16 * hf + 4 * i + 1], ov[16 * hf + 4 * i + 2],
                                             ov[16 * hf + 4 * i + 3]);
            flush(D * 4, cb * 4 + 64 * hf);
          }
        }
      }
      // a NaN value was stored as zero: the warp looks at the scales of the segment's values again, and each
      // row gets its NaN in the blocks of those that it sees
      if (*zeroed != 0u) {
        uint32_t nan_blocks = 0u;
        const unsigned long long bh = w.row / static_cast<unsigned>(R);
        const int b = static_cast<int>(bh / static_cast<unsigned>(p.c.H));
        const int h = static_cast<int>(bh % static_cast<unsigned>(p.c.H));
        const int* table = p.c.block_table + static_cast<long long>(b) * p.c.max_pages;
        const int behind = min(w.len, w.kt1 * 128);
        for (int k0 = w.kt0 * 128; k0 < behind; k0 += 32) {
          const int key = k0 + lane;
          uint32_t mine = 0u, at;
          if (key < behind && kv4_row(p.c, table[key >> p.c.page_shift], h, key, at))
            mine = kv4_nan_blocks<D>(p.c.sf[1], at);
          for (uint32_t rest = __ballot_sync(0xffffffffu, mine != 0u); rest != 0u; rest &= rest - 1u) {
            const int s = __ffs(rest) - 1;
            const uint32_t theirs = __shfl_sync(0xffffffffu, mine, s);
            if (k0 + s <= lim) nan_blocks |= theirs;
          }
        }
        if (!whole || write) {
          for (; nan_blocks != 0u; nan_blocks &= nan_blocks - 1u) {
            const int at = 16 * (__ffs(nan_blocks) - 1);
            for (int i = 0; i < 16; ++i) {
              if (whole) reinterpret_cast<uint16_t*>(p.o)[(qrow0 + lane) * D + at + i] = 0x7FFFu;
              else p.part_o[prow * D + at + i] = __int_as_float(0x7FC00000);
            }
          }
        }
      }
      if constexpr (C::PAIR) {
        tc_fence_before();
        mbar_arrive(xch_empty);
      }
      if (!whole) p.part_ml[prow] = make_float2(m_run, l_run);
      else if (p.lse != nullptr && write)
        p.lse[qrow0 + lane] = l_run == 0.f ? -INFINITY : (m_run + __log2f(l_run)) * 0.69314718055994531f;
      free_segment(sg);
    }
    cp_async_wait<0>();
    if (!ok) record_timeout();
  }

  // ---- teardown: every TMEM access and MMA of this CTA is complete here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::MMA_WARP) tmem_dealloc(tmem_base, C::TMEM_COLS);
}

}  // namespace attn
