// kv4_attn_kernel.cuh - attention over the 4-bit cache for few query rows per cached head
// (include/kv4_b200.h): decoding steps, where the cache's bytes are all that counts.
//
// For one (sequence b, cached head h) the G = Hq / Hkv query heads times N query tokens are
// R = G N rows that see the same keys; they are taken in blocks of 8 NT rows. With K^ and V^ the
// values the codes stand for, the kernel computes S^T = K^ Q^T and O^T = V^^T P^T (keys, and then
// channels, on the 16-wide M side of mma.m16n8k16, the rows on the 8-wide N side), so that no
// tensor-core work is spent on rows that do not exist and the accumulators of a row are scalars
// of a lane: with g = lane / 4, t = lane % 4, a lane holds rows 2 t, 2 t + 1 of every row tile.
//  * A lane takes the codes it needs as whole vectors: of key g the D / 4 consecutive channels
//    [D/4 t, D/4 (t+1)) for S (the order of channels in a dot product is free, and q is loaded in the
//    same order), and for P V of four keys the D / 8 channels [D/8 g, D/8 (g+1)) (the order of rows in
//    O^T is free too).
//  * E2M1 codes become f16 pairs with one conversion per byte and one multiplication by the block
//    scale, both exact. For V the nibbles of two keys are first interleaved (a shift and a bit
//    select per four pairs), since P V pairs values along the keys.
//  * P leaves S^T with the keys along lanes' groups and is needed with the keys along t: one
//    movmatrix per 8 keys x 8 rows.
// Every warp streams its own 32 keys of each 256-key tile through a ring of cp.async stages (a
// 16-key group is contiguous in its page: nine 16-byte copies per lane and step, two address
// computations per group and tensor; bulk copies issued by eight lanes cost more instructions,
// since each lane's copy is issued in turn) and keeps its own running maximum, sum and O; warps meet
// only where a segment ends. What is subtracted moves only when a score exceeds it by more than 15 (log2
// units), and then to 7 below that score (kv4_below), so most steps cost one vote and no reduction across lanes, and
// a row's largest P lies between 2^7 and 2^15: inside f16, with the binades below it left to small
// probabilities (a row with one key far above the rest has thousands of them: with the maximum itself
// subtracted, P below 2^-25 were lost from O but not from the sum). They keep 11 bits down to 2^-21 of the row's largest and
// none is lost above 2^-32 of it.
//
// Schedule: the 256-key tiles of all (b, h, row block) make one long list that is cut into
// runs, one per CTA (Kv4Runs), so uneven lengths balance without the host knowing them. A run
// that covers part of a (b, h, row block) writes its unnormalised O, maximum and sum to the
// workspace (two slots per CTA: a run's first and last item); kv4_join_sm100 joins the parts in
// the order of the runs, so results do not depend on timing. It is launched with programmatic
// serialisation, so that its launch hides under the main kernel. (A join by the CTA that takes
// the item's last ticket, without a second kernel, was slower: its fence and atomic stand in every split
// segment's way, 18.4 against 14.4 us on 6 sequences of up to 2047 keys x 12 heads.)
//
// Bound: HBM at 4.5 bits a value is 12e12 values / s, 41 per SM and clock; a value costs half a
// conversion and half a multiplication (64 lanes / clk / SM each), and with everything else 2.2
// instructions of a lane. Measured (32 sequences of 32768 keys x 8 heads, d = 128, one token, 4 query heads to a key
// head): 220 us, 5.5 TB/s of the cache's bytes, 0.84 of the measured copy rate, at 62 % of the issue slots;
// after a second under the power cap (1.77 instead of 1.965 GHz) 260 us. Small batches spend their time around the
// steps. Clock stamps, us after the wait for the kernel before, inputs out of L2: one sequence of 509 keys: lengths read
// 0.7, segment found 1.8, first copies issued 2.7, q ready 3.6, first stage there 3.7, its one step done 5.7, written 7.0,
// next kernel past its wait 7.9; 16 sequences of up to 4096 keys (mean of 296 CTAs): 1.0, 2.1, 4.5, 6.4, 6.5, and the CTAs
// end between 16 and 20; the join's wait ends 1.0 later and the join itself takes 3.4 (23.0 us a call for 8.1 us of bytes).
#pragma once

#include "kv4_cache_kernel.cuh"

namespace attn {

constexpr int kDecWarps = 8;
constexpr int kDecKeys = 32;                       // keys of a warp's step
constexpr int kDecTile = kDecWarps * kDecKeys;     // 256
constexpr int kDecSegmentTiles = 2, kDecJoinTiles = 2;   // what the cut counts with: see Kv4Runs

template <int D_, int NT_>
struct Kv4DecCfg {
  static constexpr int D = D_, NT = NT_, ROWS = 8 * NT;
  static constexpr int CODE_ROW = D / 2, SF_ROW = D / 16;
  static constexpr int CTAS_PER_SM = NT == 1 ? 2 : 1;
  static constexpr int STAGES = (NT == 1 ? 3 : 6) * (D == 64 ? 2 : 1);
  // a stage of one warp: key codes, value codes, key scales, value scales
  static constexpr int ST_VC = kDecKeys * CODE_ROW, ST_KS = 2 * kDecKeys * CODE_ROW,
                       ST_VS = ST_KS + kDecKeys * SF_ROW, STAGE = ST_VS + kDecKeys * SF_ROW;
  static constexpr int RING = kDecWarps * STAGES * STAGE;
  // where a segment ends, a warp leaves its O in NT free stages of its ring, 8 rows in each, while the
  // next segment's first copies fill the others
  static constexpr int O_LD = D + 8;               // floats between rows of a warp's O
  static_assert(8 * O_LD * 4 <= STAGE && STAGES >= NT + 2, "merge stages");
  static constexpr int SMEM_ML = RING;             // [warps][ROWS] (max, sum)
  static constexpr int KSTEPS = D / 16;
  static constexpr int SMEM_NAN = SMEM_ML + kDecWarps * ROWS * 8;   // a word per thread: see nan_rows
  static constexpr int SMEM_BYTES = SMEM_NAN + kDecWarps * 32 * 4;
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 233472, "shared memory per SM");
};

// An item's (a unit's) first part, as the CTA that wrote it leaves it for the join.
struct Kv4Head {
  int parts;                 // 0: this CTA has none
  int b, h, rb, slot;        // rb: row block
};

struct Kv4AttnParams {
  Kv4Cache c;
  const uint8_t* q;          // [B, Hq, N, d]
  uint8_t* o;
  float* lse;                // or nullptr
  const int* q_lens;         // or nullptr
  float* part_o;             // workspace: [2 ctas][ROWS][D]
  float2* part_ml;           // [2 ctas][ROWS] (the value subtracted, in log2 units; sum)
  Kv4Head* heads;            // [ctas]
  int Hq, N, causal;
  int row_blocks;            // ceil(Hq / Hkv * N / ROWS)
  int ctas;                  // CTAs of the main kernel (at most; see kv4_runs)
  float scale_log2;          // scale * log2(e) * 2^k_exp
};

__device__ __forceinline__ int kv4_qlen(const Kv4AttnParams& p, int b) {
  return p.q_lens != nullptr ? kv4_clamp(p.q_lens[b], p.N) : p.N;
}
// Tiles of one (head, row block) of sequence b.
__device__ __forceinline__ int kv4_tiles(const Kv4AttnParams& p, int b) {
  return kv4_qlen(p, b) == 0 ? 0 : (kv4_len(p.c, b) + kDecTile - 1) / kDecTile;
}

// The cut of the tiles into runs, one a CTA. A further item of a run costs its CTA about kDecSegmentTiles tiles (the
// pipeline drains, results meet, q is read), and items that are cut cost the join about kDecJoinTiles.
//   * Whole items, k a CTA, if their longest run is no longer than an even cut's with the join: an item counts as
//     `whole` tiles whatever its length.
//   * Else an even cut, in which an item counts as lead + T tiles, its first `lead` without work, where runs are long
//     enough for it to matter (four tiles each; below, lead = 0).
// Measured (d = 128, 32 query heads on 8, one query): 64 sequences of 1000 keys 29.6 us in whole items, 32.2 in an even
// cut; 8 of 700 keys 9.3 and 10.7; 8 of 1000 keys (an even cut) 11.4, whole 10.9, but 32 of 1000 keys x 1 head 9.8 and
// 10.9; 12 of 4096 keys (an even cut) 23.1 with the leads, 24.8 without; one of 4096 keys 14.0 without, 15.2 with them.
// CTA c of n takes the units [start(c), start(c + 1)). (Host: fewer than 2^31.)
struct Kv4Runs {
  uint32_t units, base, rem;
  int n, lead, whole;
  __device__ __forceinline__ Kv4Runs(uint32_t tiles, uint32_t items, uint32_t longest, uint32_t ctas) {
    const uint32_t even = (tiles + items * kDecSegmentTiles) / ctas, k = (items + ctas - 1) / ctas;
    if (k * (longest + kDecSegmentTiles) <= even + kDecSegmentTiles + kDecJoinTiles) {
      lead = 0;
      whole = static_cast<int>(longest);
      units = items * longest;
      n = k > 0 ? static_cast<int>((items + k - 1) / k) : 0;
      base = k * longest;
      rem = 0;
    } else {
      lead = tiles >= 4 * ctas ? kDecSegmentTiles : 0;
      whole = 0;
      units = tiles + items * static_cast<uint32_t>(lead);
      n = static_cast<int>(min(units, ctas));
      base = units / static_cast<uint32_t>(n);
      rem = units - base * static_cast<uint32_t>(n);
    }
  }
  __device__ __forceinline__ uint32_t start(int c) const {
    return min(base * c + min(static_cast<uint32_t>(c), rem), units);
  }
  __device__ __forceinline__ int cta_of(uint32_t u) const {
    const uint32_t longer = rem * (base + 1u);
    return static_cast<int>(u < longer ? u / (base + 1u) : rem + (u - longer) / base);
  }
  __device__ __forceinline__ uint32_t item_units(int T) const {   // of an item of T > 0 tiles
    return static_cast<uint32_t>(max(T + lead, whole));
  }
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ uint32_t warp_prefix(uint32_t v, int lane) {     // inclusive
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// 16-byte asynchronous copy global -> shared; with `valid` false nothing is read and zeros are written
__device__ __forceinline__ void cp_async_16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const uint8_t* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// a f16x2 of one half of x
__device__ __forceinline__ uint32_t splat_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t splat_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma_16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 0xFF for each of the four scale bytes that is a NaN
__device__ __forceinline__ uint32_t nan_scales(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// Blocks of a value row (its number in the cache) whose scale is a NaN, a bit each.
template <int D>
__device__ __forceinline__ uint32_t kv4_nan_blocks(const uint8_t* sf, uint32_t row) {
  uint32_t blocks = 0u;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(sf + static_cast<size_t>(row) * (D / 16))[i];
    blocks |= (((nan_scales(w) & 0x01010101u) * 0x01020408u) >> 24) << (4 * i);   // the product gathers the four bits
  }
  return blocks;
}

constexpr float kPShift = 7.f, kPRoom = 8.f;         // log2 of the largest P where the subtracted value is set, and its growth
// The value that is subtracted for a row whose largest score so far (log2 units) is x, and when a score is out of reach.
__device__ __forceinline__ float kv4_below(float x) { return x - kPShift; }
__device__ __forceinline__ bool kv4_outgrown(float x, float m) { return x > m + (kPShift + kPRoom); }

// A query row's exponent: q 2^-e lies below 2^10 in magnitude and its largest value at or above 2^9
// (rows of zeros and of very small values: as far as an fp32 power of two goes; a row with an
// infinity or NaN is left as it is). Returns the exponent field of 2^e.
__device__ __forceinline__ int kv4_row_exp(float amax) {
  const int ef = static_cast<int>(__float_as_uint(amax) >> 23);
  return ef == 255 ? 127 : max(ef, 10) - 9;
}

// O = 0, LSE = -infinity for the rows that see no key.
template <int D>
__device__ __forceinline__ void kv4_empty_rows(const Kv4AttnParams& p, int thread, int threads) {
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
    const int len = kv4_len(p.c, b), n = kv4_qlen(p, b);
    const int z = len == 0 ? n : (p.causal ? max(0, n - len) : 0);
    if (z == 0) continue;
    constexpr int V4 = D / 8;                        // 16-byte pieces of a row
    for (long long i = thread; i < static_cast<long long>(p.Hq) * z * V4; i += threads) {
      const long long r = i / V4;
      const size_t row = (static_cast<size_t>(b) * p.Hq + r / z) * p.N + r % z;
      reinterpret_cast<uint4*>(p.o)[row * V4 + i % V4] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr && i % V4 == 0) p.lse[row] = -INFINITY;
    }
  }
}

// What a row's unnormalised O is multiplied with. A sum of zero is that of a row without keys (O = 0), or of one
// whose every score is -infinity (from a query that is infinite: NaN).
__device__ __forceinline__ float kv4_norm(const Kv4AttnParams& p, float L, bool sees) {
  return L != 0.f ? f32_exp2i(p.c.exp[1]) / L : sees ? __int_as_float(0x7FC00000) : 0.f;
}

// One row's result from its unnormalised O (4 channels a lane at d4), maximum and sum.
template <int D, bool F16>
__device__ __forceinline__ void kv4_write_row(const Kv4AttnParams& p, size_t row, int d4, float4 a, float M, float L, bool sees) {
  const float inv = kv4_norm(p, L, sees);
  reinterpret_cast<uint2*>(p.o)[row * (D / 4) + d4] =
      make_uint2(pack_16<F16>(a.x * inv, a.y * inv), pack_16<F16>(a.z * inv, a.w * inv));
  if (p.lse != nullptr && d4 == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

template <class C, bool F16>
__global__ void __launch_bounds__(kDecWarps * 32, C::CTAS_PER_SM) kv4_decode_sm100(const Kv4AttnParams p) {
  constexpr int D = C::D, NT = C::NT, ROWS = C::ROWS;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t smem0 = b200::smem_addr(smem_raw);
  kv4_grid_wait();
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) p.heads[blockIdx.x].parts = 0;
  const uint32_t ring = smem0 + warp * C::STAGES * C::STAGE;

  // Copies. Codes: lane takes bytes [16 lane, 16 lane + 16) of every 512 of a group's. Scales: lane
  // takes 16 bytes of (tensor, group, piece); `grp` is also the group whose page it looks up.
  constexpr int SFP = C::SF_ROW;                    // 16-byte pieces of a group's scales (16 rows)
  const int grp = (lane / SFP) & 1;
  const uint8_t* kptr = p.c.codes[0] + lane * 16;
  const uint8_t* vptr = p.c.codes[1] + lane * 16;
  const uint8_t* sptr = p.c.sf[(lane / (2 * SFP)) & 1] + (lane % SFP) * 16;
  asm volatile("" : "+l"(kptr), "+l"(vptr), "+l"(sptr));    // kept in registers
  const uint32_t kdst = ring + lane * 16;
  const uint32_t sdst = ring + ((lane / (2 * SFP)) & 1 ? C::ST_VS : C::ST_KS) + (grp * SFP + lane % SFP) * 16;
  const bool scopy = lane < 4 * SFP;
  // S^T row g of an 8-row group is key g, with 2, 3 and 6, 7 swapped: K's 16-byte loads (two rows a
  // phase) stay free of bank conflicts and V's 8-byte loads of the keys of rows 2 t meet two to
  // a bank instead of four
  const int gk = g ^ ((g >> 1) & 1), va = 2 * t + (t & 1), vb = 2 * t + 1 - (t & 1);
  // this CTA's run, and the (sequence, tiles before it) where it starts. Up to 32 sequences' lengths
  // stay in the lanes; more are read again.
  const int per_b = p.c.H * p.row_blocks;
  const bool few = p.c.B <= 32;
  int my_len = 0, my_n = 0, my_T = 0;                         // of sequence `lane`, if few
  uint32_t tiles = 0, items = 0, longest = 0;
  bool blind = false;                               // some row sees no key
  for (int i = lane; i < p.c.B; i += 32) {
    my_len = kv4_len(p.c, i);
    my_n = kv4_qlen(p, i);
    const uint32_t T = my_n == 0 ? 0u : static_cast<uint32_t>(my_len + kDecTile - 1) / kDecTile;
    tiles += T * per_b;
    items += T > 0u ? per_b : 0u;
    longest = max(longest, T);
    my_T = static_cast<int>(T);
    blind = blind || (my_n > 0 && (my_len == 0 || (p.causal && my_n > my_len)));
  }
  if (__any_sync(0xffffffffu, blind)) kv4_empty_rows<D>(p, tid, kDecWarps * 32);
  const Kv4Runs runs(warp_sum(tiles), warp_sum(items), __reduce_max_sync(0xffffffffu, longest), p.ctas);
  if (static_cast<int>(blockIdx.x) >= runs.n) return;
  uint32_t u = runs.start(blockIdx.x);
  const uint32_t u_end = runs.start(blockIdx.x + 1);
  auto units_of = [&](int T) { return T > 0 ? runs.item_units(T) * per_b : 0u; };
  int b = 0;
  uint32_t b_first = 0;                             // first unit of sequence b
  for (int b0 = 0;; b0 += 32) {
    const uint32_t mine = b0 + lane < p.c.B ? units_of(few ? my_T : kv4_tiles(p, b0 + lane)) : 0u;
    const uint32_t incl = warp_prefix(mine, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, b_first + incl > u);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      b_first += __shfl_sync(0xffffffffu, incl - mine, l);
      break;
    }
    b_first += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int R = p.Hq / p.c.H * p.N;
  const uint32_t slot_mask = (1u << p.c.page_shift) - 1u, page_rows = static_cast<uint32_t>(p.c.H) << p.c.page_shift;

  // the segment being worked on: tiles [t0, t1) of T of (b, h, row block rb)
  int T, h, rb, t0, t1, len, n, steps_end, base0;
  uint32_t hrow;
  uint32_t item_first;                              // its item's first tile, as a unit
  size_t row0;                                      // rows of (b, h) are contiguous in q and o
  const int* table;
  auto find_segment = [&]() {                       // the first with work at or after unit u; moves u behind it
    while (u < u_end) {
      len = few ? __shfl_sync(0xffffffffu, my_len, b) : kv4_len(p.c, b);
      n = few ? __shfl_sync(0xffffffffu, my_n, b) : kv4_qlen(p, b);
      T = n == 0 ? 0 : (len + kDecTile - 1) / kDecTile;
      if (u >= b_first + units_of(T)) {
        b_first += units_of(T);
        ++b;
        continue;
      }
      const uint32_t per = runs.item_units(T), item = (u - b_first) / per;
      item_first = b_first + (item + 1u) * per - static_cast<uint32_t>(T);
      h = static_cast<int>(item) / p.row_blocks, rb = static_cast<int>(item) % p.row_blocks;
      t0 = max(0, static_cast<int>(u - item_first));
      t1 = min(T, static_cast<int>(u_end - item_first));
      u = item_first + max(t1, 0);
      if (t1 <= t0) return false;                   // the run ends before the item's first tile
      row0 = (static_cast<size_t>(b) * p.c.H + h) * R;
      table = p.c.block_table + static_cast<long long>(b) * p.c.max_pages;
      steps_end = min(t1 * kDecTile, len);          // its keys end here
      base0 = t0 * kDecTile + warp * kDecKeys;      // this warp's first step
      hrow = static_cast<uint32_t>(h) << p.c.page_shift;
      return true;
    }
    return false;
  };

  // ---- a warp's pipeline over its 32-key steps
  auto page_of = [&](int base) {                  // page of this lane's group
    const int key = base + 16 * grp;
    return key < steps_end ? static_cast<uint32_t>(table[key >> p.c.page_shift]) : 0u;
  };
  auto issue = [&](int base, uint32_t st, uint32_t pg) {
    if (base < steps_end) {
      const int key = base + 16 * grp;
      const uint32_t row = pg * page_rows + (hrow + (static_cast<uint32_t>(key) & slot_mask));
      if (__all_sync(0xffffffffu, pg < static_cast<uint32_t>(p.c.num_pages) && base + kDecKeys <= steps_end)) {
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const uint32_t rr = __shfl_sync(0xffffffffu, row, gr * SFP);
          const uint8_t* ks = kptr + static_cast<size_t>(rr) * C::CODE_ROW;
          const uint8_t* vs = vptr + static_cast<size_t>(rr) * C::CODE_ROW;
#pragma unroll
          for (int i = 0; i < 16 * C::CODE_ROW; i += 512) {
            cp_async_16(kdst + st + gr * 16 * C::CODE_ROW + i, ks + i);
            cp_async_16(kdst + st + C::ST_VC + gr * 16 * C::CODE_ROW + i, vs + i);
          }
        }
        if (scopy) cp_async_16(sdst + st, sptr + static_cast<size_t>(row) * C::SF_ROW);
      } else {
        // a sequence's last step, or a page outside the cache: what is not there is zero (keys behind
        // the end inside a copied group are masked, and their scales looked at, below)
        uint32_t unused;
        const bool mine = key < steps_end && kv4_row(p.c, static_cast<int>(pg), h, key, unused);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const bool v = __shfl_sync(0xffffffffu, mine, gr * SFP);
          const uint32_t rr = __shfl_sync(0xffffffffu, mine ? row : 0u, gr * SFP);
#pragma unroll
          for (int i = 0; i < 16 * C::CODE_ROW; i += 512) {
            cp_async_16z(kdst + st + gr * 16 * C::CODE_ROW + i, kptr + static_cast<size_t>(rr) * C::CODE_ROW + i, v);
            cp_async_16z(kdst + st + C::ST_VC + gr * 16 * C::CODE_ROW + i,
                         vptr + static_cast<size_t>(rr) * C::CODE_ROW + i, v);
          }
        }
        if (scopy) cp_async_16z(sdst + st, sptr + static_cast<size_t>(mine ? row : 0u) * C::SF_ROW, mine);
      }
    }
    cp_async_commit();
  };
  auto after = [](uint32_t st) { return st == (C::STAGES - 1) * C::STAGE ? 0u : st + C::STAGE; };
  uint32_t rd = 0, wr = 0;                          // offsets of the stage to use and of the one to fill
  uint32_t page = 0;                                // of the step to issue next
  int next_base = 0;
  auto issue_next = [&](int count) {
    for (int i = 0; i < count; ++i) {
      const uint32_t nx = page_of(next_base + kDecTile);
      issue(next_base, wr, page);
      page = nx;
      next_base += kDecTile;
      wr = after(wr);
    }
  };
  auto start_segment = [&](int stages) {            // its first copies
    next_base = base0;
    page = page_of(base0);
    issue_next(stages);
  };
  // q: lane (g, t) takes channels [D/4 t, D/4 (t+1)) of row g of each tile
  // (NT = 1: loaded ahead, under the copies' latency)
  constexpr bool AHEAD = NT == 1;
  uint32_t qw[D / 8];
  auto load_q = [&](int nt) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int r = rb * ROWS + nt * 8 + g;
      const uint4 x = r < R ? reinterpret_cast<const uint4*>(p.q + ((row0 + r) * D + t * (D / 4)) * 2)[i]
                            : make_uint4(0u, 0u, 0u, 0u);
      qw[4 * i] = x.x, qw[4 * i + 1] = x.y, qw[4 * i + 2] = x.z, qw[4 * i + 3] = x.w;
    }
  };

  if (!find_segment()) return;
  bool first_segment = true;
  start_segment(C::STAGES - 1);
  if (AHEAD) load_q(0);
  for (;;) {
    // ---- q fragments
    uint32_t qf[NT][C::KSTEPS][2];
    float cs[NT][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!AHEAD) load_q(nt);
      uint32_t (&w)[D / 8] = qw;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 f = f32x2_from_16<F16>(w[i]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = kv4_row_exp(amax);
      const float down = __int_as_float((254 - e) << 23), up = __int_as_float(e << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 f = f32x2_from_16<F16>(w[i]);
        w[i] = b200::pack_f16x2(f.x * down, f.y * down);
      }
#pragma unroll
      for (int k = 0; k < C::KSTEPS; ++k) {
        qf[nt][k][0] = w[2 * k];
        qf[nt][k][1] = w[2 * k + 1];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // (kept above zero: a masked score is -infinity and has to stay that)
        cs[nt][j] = fmaxf(__shfl_sync(0xffffffffu, up, 4 * (2 * t + j)) * p.scale_log2, 1e-37f);
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
    }
    const int lim_all = p.causal ? len - n : len - 1;       // every row sees the keys up to here
    // bits 2 nt + j: this lane's rows and channels that a NaN value belongs in which the product takes as zero (see the
    // masks; in shared memory, since it is rare: O made NaN in the step itself cost 2 % on 32 sequences of 32768 keys)
    uint32_t* const nan_rows = reinterpret_cast<uint32_t*>(smem_raw + C::SMEM_NAN) + tid;
    *nan_rows = 0u;
    float o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;

    for (int base = base0; base < steps_end; base += kDecTile) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      const uint32_t nx = page_of(base + C::STAGES * kDecTile);
      issue(base + (C::STAGES - 1) * kDecTile, wr, page);
      page = nx;
      wr = rd;                                      // the stage to fill is the one used last
      const uint8_t* st = smem_raw + (ring - smem0) + rd;
      rd = after(rd);
      // ---- S^T of 32 keys
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t kw[2][D / 32];                     // codes of keys (S^T rows) g and g + 8
        uint32_t ks[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int slot = 16 * mt + 8 * j + gk;
          const uint8_t* a = st + slot * C::CODE_ROW + t * (D / 8);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(a);
            kw[j][0] = x.x, kw[j][1] = x.y, kw[j][2] = x.z, kw[j][3] = x.w;
            ks[j] = b200::f16x2_from_e4m3x2(*reinterpret_cast<const uint16_t*>(st + C::ST_KS + slot * 8 + 2 * t));
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(a);
            kw[j][0] = x.x, kw[j][1] = x.y;
            const uint32_t by = st[C::ST_KS + slot * 4 + t];
            ks[j] = b200::f16x2_from_e4m3x2(static_cast<uint16_t>(by | (by << 8)));
          }
        }
#pragma unroll
        for (int wd = 0; wd < D / 32; ++wd) {       // a word: 8 channels, two k-steps
          uint32_t f[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f16x2_from_e2m1x8(kw[j][wd], f[j]);
            const uint32_t sc = D == 128 ? (wd < 2 ? splat_lo(ks[j]) : splat_hi(ks[j])) : ks[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[j][i] = hmul2(f[j][i], sc);
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t a[4] = {f[0][2 * hf], f[1][2 * hf], f[0][2 * hf + 1], f[1][2 * hf + 1]};
            const int k = 2 * wd + hf;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (k == 0)
                mma_16816_zero(s[mt][nt], a, qf[nt][k][0], qf[nt][k][1]);
              else
                mma_16816(s[mt][nt], a, qf[nt][k][0], qf[nt][k][1]);
            }
          }
        }
      }
      // ---- masks: only steps that some row does not see to their end
      uint32_t vnan = 0u;                           // (masked steps) keys whose values hold a NaN
      if (base + kDecKeys - 1 > lim_all) {
        bool bad;
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(st + C::ST_VS + lane * 8);
          bad = (nan_scales(x.x) | nan_scales(x.y)) != 0u;
        } else {
          bad = nan_scales(*reinterpret_cast<const uint32_t*>(st + C::ST_VS + lane * 4)) != 0u;
        }
        vnan = __ballot_sync(0xffffffffu, bad);
        auto limit = [&](int nt, int j) {           // a row's last visible key, from `base`
          const int rr = rb * ROWS + nt * 8 + 2 * t + j;
          return (p.causal ? len - n + rr % p.N : len - 1) - base;
        };
        // P = 0 would not keep a NaN value from a row that does not see it: such values count as zero in this
        // step (below), and the rows that see them are noted: their O becomes NaN where the segment ends (a lane's
        // channels lie in one block; rows see prefixes, so the first such key decides)
        if (vnan != 0u) {
          int first = kDecKeys;
          for (uint32_t rest = vnan; rest != 0u; rest &= rest - 1u) {
            const int k = __ffs(rest) - 1;
            if ((st[C::ST_VS + k * C::SF_ROW + g * C::SF_ROW / 8] & 0x7Fu) == 0x7Fu) first = min(first, k);
          }
          if (first < kDecKeys) {
            uint32_t rows = 0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) rows |= first <= limit(nt, j) ? 1u << (2 * nt + j) : 0u;
            *nan_rows |= rows;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int lim = limit(nt, j);
#pragma unroll
            for (int i = 0; i < 4; ++i)             // 8 i + gk: the key of this S^T row
              if (8 * i + gk > lim) s[i >> 1][nt][2 * (i & 1) + j] = -INFINITY;
          }
      }
      // ---- online softmax
      bool grow = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[nt][j] = cs[nt][j] * fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]), fmaxf(s[1][nt][j], s[1][nt][j + 2]));
          grow = grow || kv4_outgrown(mx[nt][j], m[nt][j]);
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = mx[nt][j];
#pragma unroll
            for (int sft = 4; sft < 32; sft <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sft));
            const float mn = fmaxf(m[nt][j], kv4_below(x));
            const float al = mn == -INFINITY ? 1.f : b200::ex2_approx(m[nt][j] - mn);
            m[nt][j] = mn;
            l[nt][j] *= al;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][j] *= al;
              o[nt][i][j + 2] *= al;
            }
          }
      }
      uint32_t pb[2][NT][2];                        // P^T fragments: keys 2 t (+1), and + 8, of each 16-key tile
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p0 = b200::ex2_approx(fmaf(s[mt][nt][2 * hf], cs[nt][0], -m0));
            const float p1 = b200::ex2_approx(fmaf(s[mt][nt][2 * hf + 1], cs[nt][1], -m1));
            l[nt][0] += p0;
            l[nt][1] += p1;
            pb[mt][nt][hf] = movmatrix(b200::pack_f16x2(p0, p1));
          }
      }
      // ---- O^T += V^^T P^T over the keys of S^T rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t vw[4][D / 64];
        uint32_t by[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * mt + 8 * (i >> 1) + ((i & 1) ? vb : va);
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(st + C::ST_VC + r * 64 + g * 8);
            vw[i][0] = x.x, vw[i][1] = x.y;
            by[i] = st[C::ST_VS + r * 8 + g];
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(st + C::ST_VC + r * 32 + g * 4);
            by[i] = st[C::ST_VS + r * 4 + (g >> 1)];
          }
        }
        if (vnan != 0u) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((by[i] & 0x7Fu) == 0x7Fu) by[i] = 0u;
        }
        uint32_t vs[2];
#pragma unroll
        for (int pr = 0; pr < 2; ++pr)
          vs[pr] = b200::f16x2_from_e4m3x2(static_cast<uint16_t>(by[2 * pr] | (by[2 * pr + 1] << 8)));
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          uint32_t ev[2][4], od[2][4];              // f16 pairs (two keys) of even and odd channels
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const uint32_t wa = vw[2 * pr][wd], wb = vw[2 * pr + 1][wd];
            f16x2_from_e2m1x8((wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u), ev[pr]);
            f16x2_from_e2m1x8(((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u), od[pr]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ev[pr][i] = hmul2(ev[pr][i], vs[pr]);
              od[pr][i] = hmul2(od[pr][i], vs[pr]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a[4] = {ev[0][i], od[0][i], ev[1][i], od[1][i]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][4 * wd + i], a, pb[mt][nt][0], pb[mt][nt][1]);
          }
        }
      }
    }
    // ---- the segment ends: the next one's first copies go out, and the warps' results meet in shared
    // memory. Copies that the loop issued past the segment's end were empty, so `rd` is the next stage.
    cp_async_wait<0>();
    __syncwarp();
    if (base0 + (t1 - t0 - 1) * kDecTile >= steps_end) rd = after(rd);   // the last tile ends before this warp's
                                                    // keys: every warp's ring stands at the same stage
    const bool whole = t0 == 0 && t1 == T;
    const int slot = 2 * blockIdx.x + (first_segment ? 0 : 1);
    first_segment = false;
    const int out_rb = rb, out_n = n, out_blind = p.causal ? n - len : 0;   // queries before out_blind see no key
    if (tid == 0 && t0 == 0 && !whole) {            // the item's first part: what the join needs
      Kv4Head hd;
      hd.parts = runs.cta_of(item_first + T - 1) - static_cast<int>(blockIdx.x) + 1;
      hd.b = b, hd.h = h, hd.rb = rb, hd.slot = slot;
      p.heads[blockIdx.x] = hd;
    }
    const size_t out_row0 = row0;
    wr = rd;
    const bool more = find_segment();
    if (more) {
      start_segment(C::STAGES - NT);
    } else {
      for (int i = 0; i < C::STAGES - NT; ++i) wr = after(wr);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int sft = 4; sft < 32; sft <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], sft);
    float2* ml = reinterpret_cast<float2*>(smem_raw + C::SMEM_ML);
    uint32_t mst[NT];                               // the stages that take O
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mst[nt] = nt == 0 ? wr : after(mst[nt > 0 ? nt - 1 : 0]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 2 * t + j;
        if (g == 0) ml[warp * ROWS + nt * 8 + r] = make_float2(m[nt][j], l[nt][j]);
        float* dst = reinterpret_cast<float*>(smem_raw + warp * C::STAGES * C::STAGE + mst[nt]) + r * C::O_LD + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<float4*>(dst + 4 * i) =
              make_float4(o[nt][2 * i][j], o[nt][2 * i][j + 2], o[nt][2 * i + 1][j], o[nt][2 * i + 1][j + 2]);
      }
    if (const uint32_t bits = *nan_rows; bits != 0u) {
      for (int x = 0; x < 2 * NT; ++x) {
        if (((bits >> x) & 1u) == 0u) continue;
        float* dst = reinterpret_cast<float*>(smem_raw + warp * C::STAGES * C::STAGE + (x < 2 ? mst[0] : mst[NT - 1])) +
                     (2 * t + (x & 1)) * C::O_LD + g * (D / 8);
        for (int i = 0; i < D / 8; ++i) dst[i] = __int_as_float(0x7FC00000);
      }
    }
    if (AHEAD && more) load_q(0);
    __syncthreads();
    constexpr int V4 = D / 4;                       // float4 per row
    for (int i = tid; i < ROWS * V4; i += kDecWarps * 32) {
      const int r = i / V4, d4 = i % V4;
      uint32_t mst_r = mst[0];
#pragma unroll
      for (int nt = 1; nt < NT; ++nt)
        if ((r >> 3) == nt) mst_r = mst[nt];
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * ROWS + r].x);
      const float Mu = M == -INFINITY ? 0.f : M;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 x = ml[w * ROWS + r];
        const float f = b200::ex2_approx(x.x - Mu);
        const float4 v = *reinterpret_cast<const float4*>(smem_raw + w * C::STAGES * C::STAGE + mst_r + ((r & 7) * C::O_LD + 4 * d4) * 4);
        L += f * x.y;
        a.x += f * v.x, a.y += f * v.y, a.z += f * v.z, a.w += f * v.w;
      }
      if (whole) {
        const int rr = out_rb * ROWS + r;
        if (rr < R && rr % p.N < out_n) {
          kv4_write_row<D, F16>(p, out_row0 + rr, d4, a, M, L, rr % p.N >= out_blind);
        }
      } else {
        reinterpret_cast<float4*>(p.part_o)[(static_cast<size_t>(slot) * ROWS + r) * V4 + d4] = a;
        if (d4 == 0) p.part_ml[static_cast<size_t>(slot) * ROWS + r] = make_float2(M, L);
      }
    }
    if (!more) return;
    __syncthreads();
    if constexpr (NT > 1) issue_next(NT - 1);
  }
}

// Joins the parts of the item whose first part CTA blockIdx.x wrote (row blocks of ROWS rows): a warp per
// row. A lane holds the
// (maximum, sum) of one part, so that the parts' O, D / 32 channels a lane, load without waiting for
// one another.
template <int D, int ROWS, bool F16>
__global__ void __launch_bounds__(256) kv4_join_sm100(const Kv4AttnParams p) {
  constexpr int E = D / 32;
  kv4_grid_wait();
  const Kv4Head hd = p.heads[blockIdx.x];
  if (hd.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.Hq / p.c.H * p.N, n = kv4_qlen(p, hd.b);
  const int r = blockIdx.y * 8 + warp, rr = hd.rb * ROWS + r;
  if (rr >= R || rr % p.N >= n) return;
  float M = -INFINITY, L = 0.f, a[E] = {};
  for (int i0 = 0; i0 < hd.parts; i0 += 32) {
    auto at = [&](int i) {
      return static_cast<size_t>(i == 0 ? hd.slot : 2 * (static_cast<int>(blockIdx.x) + i)) * ROWS + r;
    };
    const int i = i0 + lane;
    const float2 x = i < hd.parts ? p.part_ml[at(i)] : make_float2(-INFINITY, 0.f);
    float mx = x.x;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float Mn = fmaxf(M, mx), Mu = Mn == -INFINITY ? 0.f : Mn;
    const float fo = b200::ex2_approx(M - Mu), mine = b200::ex2_approx(x.x - Mu);
    // (a part whose keys lie behind this row's has no O: nothing was written)
    const uint32_t full = __ballot_sync(0xffffffffu, !(x.x == -INFINITY && x.y == 0.f));
    float sum = x.y * mine;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    L = L * fo + sum;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] *= fo;
    const int m = min(32, hd.parts - i0);
#pragma unroll 8
    for (int k = 0; k < m; ++k) {
      const float f = __shfl_sync(0xffffffffu, mine, k);
      const bool have = (full >> k) & 1u;
      const float* src = p.part_o + at(i0 + k) * D + lane;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] += f * (have ? src[32 * e] : 0.f);
    }
    M = Mn;
  }
  const float inv = kv4_norm(p, L, L == 0.f && (!p.causal || rr % p.N >= n - kv4_len(p.c, hd.b)));
  const size_t row = (static_cast<size_t>(hd.b) * p.c.H + hd.h) * R + rr;
#pragma unroll
  for (int e = 0; e < E; ++e)
    reinterpret_cast<uint16_t*>(p.o)[row * D + lane + 32 * e] = static_cast<uint16_t>(pack_16<F16>(a[e] * inv, 0.f));
  if (p.lse != nullptr && lane == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

}  // namespace attn
