// kv4_cache_kernel.cuh - the 4-bit key/value cache: its format on the device, and the
// kernels that quantise new tokens into it and read positions back
// (include/kv4_b200.h gives the definition).
//
// A row is one token of one head: d / 2 bytes of E2M1 codes and d / 16 E4M3 scale
// bytes. Both kernels move bytes and little else: a CTA takes 64 rows of one head
// (of one tensor), its lanes consecutive pieces of a row.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100.cuh"
#include "status.cuh"

namespace attn {

// Every kernel of the cache is launched so that its CTAs may start while the kernel before it in the stream ends, and
// waits here, before it touches any memory (or allocates tensor memory), until that one is complete: the launch alone
// overlaps (6 sequences of 2047 keys x 12 heads 14.4 -> 12.3 us a call). So the kernel lives while the one before it
// may still write what it reads: inputs, tables, cache and parts are read by plain loads (or asynchronous copies) behind
// the wait, which its memory clobber holds back, and never through the read-only path (__ldg, ld.global.nc), which asks
// for memory that nothing writes while the kernel lives. (Times are the same within 1 % either way.)
__device__ __forceinline__ void kv4_grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The cache as every kernel sees it.
struct Kv4Cache {
  uint8_t* codes[2];         // keys, values: [num_pages, H, page_size, d / 2]
  uint8_t* sf[2];            // [num_pages, H, page_size, d / 16]
  const int* block_table;    // [B, max_pages]
  const int* seq_lens;       // [B]
  int B, H, num_pages, page_shift, max_pages;
  int exp[2];                // k_exp, v_exp
};

// An index that the call's device arrays put outside the cache: recorded in every
// build, and the access is skipped.
__device__ __forceinline__ void kv4_record(unsigned long long index) {
  atomicOr(&g_status, kStatusBounds);
  if constexpr (kDebugChecks) {
    if (atomicCAS(&g_debug_site, 0u, static_cast<uint32_t>(kSiteKv4Index)) == 0u) atomicExch(&g_debug_index, index);
  }
}

// x clamped to [0, hi]; a value outside is recorded.
__device__ __forceinline__ int kv4_clamp(int x, int hi) {
  if (x >= 0 && x <= hi) return x;
  kv4_record(static_cast<unsigned long long>(static_cast<long long>(x)));
  return x < 0 ? 0 : hi;
}

// Tokens of sequence b in the cache.
__device__ __forceinline__ int kv4_len(const Kv4Cache& c, int b) {
  return kv4_clamp(c.seq_lens[b], c.max_pages << c.page_shift);
}

// Row index (page, head, slot) of position `pos` given its page number; false for a page
// outside the cache.
__device__ __forceinline__ bool kv4_row(const Kv4Cache& c, int page, int h, int pos, uint32_t& row) {
  const uint32_t slot = static_cast<uint32_t>(pos) & ((1u << c.page_shift) - 1u);
  row = ((static_cast<uint32_t>(page) * static_cast<uint32_t>(c.H) + static_cast<uint32_t>(h)) << c.page_shift) + slot;
  if (static_cast<uint32_t>(page) < static_cast<uint32_t>(c.num_pages)) return true;
  kv4_record(static_cast<unsigned long long>(static_cast<uint32_t>(page)));
  return false;
}

// ---------------------------------------------------------------- conversions
// four bytes of two E2M1 codes each -> four f16x2 (low nibble in the low half; exact)
__device__ __forceinline__ void f16x2_from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// two fp32 -> one byte of two E2M1 codes (round to nearest even, saturating), lo in the low nibble
__device__ __forceinline__ uint32_t e2m1x2_from_f32(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
      "mov.b32 %0, {t, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32x2_from_f16x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float f32_exp2i(int e) { return __int_as_float((e + 127) << 23); }   // |e| <= 126

template <bool F16>
__device__ __forceinline__ float2 f32x2_from_16(uint32_t w) {
  if constexpr (F16) return f32x2_from_f16x2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi) {
  return F16 ? b200::pack_f16x2(lo, hi) : b200::pack_bf16x2(lo, hi);
}

// ---------------------------------------------------------------- kernels
constexpr int kKv4Threads = 256;
constexpr int kKv4Rows = 64;     // rows (tokens) of one (b, h) that a CTA moves
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct Kv4MoveParams {
  Kv4Cache c;
  const uint8_t* in[2];     // append: k, v [B, H, N, d] 16-bit values
  uint8_t* out[2];          // read: k, v
  const int* first;         // append: new_lens or nullptr; read: starts or nullptr
  int N, tiles;             // tiles of kKv4Rows rows per (b, h)
};

// The CTA's (b, h) and first row: blockIdx.x counts tiles of kKv4Rows rows, blockIdx.y is 0 for keys, 1
// for values. Everything here is the same for the whole CTA, so that a thread is left with one page lookup per row.
struct Kv4MoveTile {
  int b, h, i0;
  size_t row0;               // of i0 in the dense tensor
  __device__ __forceinline__ explicit Kv4MoveTile(const Kv4MoveParams& p) {
    const int bh = static_cast<int>(blockIdx.x) / p.tiles;
    i0 = (static_cast<int>(blockIdx.x) - bh * p.tiles) * kKv4Rows;
    b = bh / p.c.H;
    h = bh - b * p.c.H;
    row0 = static_cast<size_t>(bh) * p.N + i0;
  }
};

// Cache row of position pos of sequence b (kNoRow for pos < 0 and for a page outside the cache).
__device__ __forceinline__ uint32_t kv4_lookup(const Kv4MoveParams& p, int b, int h, int pos) {
  uint32_t row;
  if (pos < 0) return kNoRow;
  const int page = p.c.block_table[static_cast<long long>(b) * p.c.max_pages + (pos >> p.c.page_shift)];
  return kv4_row(p.c, page, h, pos, row) ? row : kNoRow;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// In both kernels a warp moves 8 rows: LPR lanes hold a row, 32 / LPR rows make a pass, and one lane looks up
// each of the 8 rows. Both are near the bytes they move, and instructions are what is left: with every lane
// looking up its own row, and quotients rounded in integers, a prompt (4 x 8 heads x 4096 tokens written
// and read back) took 38.0 us instead of 34.1 and a read of 8 heads x 32768 tokens 32.2 instead of 30.6 (33.9 and 29.9
// since the launches overlap).
constexpr int kKv4WarpRows = kKv4Rows / (kKv4Threads / 32);
static_assert(kKv4WarpRows == 8, "rows of a warp");

// Quantises new tokens: a thread takes one block of 16 values of each of its rows. A quotient q = y / s
// decides a code only by its side of a border of E2M1 (t = 0.25 ... 5). It is taken as y * (1 / s) rounded to
// a multiple of 2^-16 by adding and subtracting 192, which decides alike: y has at most 11 significant bits and
// t s at most 7, so q is t itself or at least 2^-11 t >= 2^-13 away from it; 1 / s is off by 2^-24 of
// itself and the sum rounds by 2^-17, so an exact t comes out as t and nothing crosses one. The sum loses the sign
// of a quotient that rounds to zero, which is put back: codes are those of the definition bit for bit. (Sixteen IEEE
// divisions a block took 2 us more on that prompt; the sums one at a time and not in pairs 0.9 us.)
template <int D, bool F16>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_sm100(const __grid_constant__ Kv4MoveParams p) {
  constexpr int LPR = D / 16, RPP = 32 / LPR, U = kKv4WarpRows / RPP;   // lanes per row, rows per pass, passes
  const int which = blockIdx.y, lane = threadIdx.x & 31, blk = lane % LPR;
  const int exp2 = which == 0 ? p.c.exp[0] : p.c.exp[1];
  kv4_grid_wait();
  const Kv4MoveTile tile(p);
  const int r0 = (threadIdx.x >> 5) * kKv4WarpRows;                     // the warp's first row of the tile
  const uint4* src = reinterpret_cast<const uint4*>(which == 0 ? p.in[0] : p.in[1]) + tile.row0 * (LPR * 2) + blk * 2;
  uint4 x[U][2];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int r = r0 + j * RPP + lane / LPR;
    if (tile.i0 + r < p.N) {
      x[j][0] = src[r * (LPR * 2)];
      x[j][1] = src[r * (LPR * 2) + 1];
    }
  }
  const int len = kv4_len(p.c, tile.b), n = p.first != nullptr ? kv4_clamp(p.first[tile.b], p.N) : p.N;
  if (n > len) kv4_record(static_cast<unsigned long long>(static_cast<long long>(len - n)));   // tokens before position 0
  const int mine = tile.i0 + r0 + (lane & 7);
  const uint32_t my_row = kv4_lookup(p, tile.b, tile.h, lane < 8 && mine < n ? len - n + mine : -1);
  uint8_t* const codes = (which == 0 ? p.c.codes[0] : p.c.codes[1]) + blk * 8;
  uint8_t* const sf = (which == 0 ? p.c.sf[0] : p.c.sf[1]) + blk;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t row = __shfl_sync(0xffffffffu, my_row, j * RPP + lane / LPR);
    if (row == kNoRow) continue;
    const uint32_t w[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
    float v[16];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = f32x2_from_16<F16>(w[k]);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
      amax = max_nan(amax, max_nan(fabsf(f.x), fabsf(f.y)));
    }
    const bool nan = amax != amax;
    const float down = f32_exp2i(-exp2);
    const float want = fminf(fmaxf(__fdiv_rn(amax * down, 6.f), 0.001953125f), 448.f);
    const uint32_t byte = b200::pack_e4m3x4(want, 0.f, 0.f, 0.f) & 0xFFu;
    const float inv = __frcp_rn(f32x2_from_f16x2(b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte))).x) * down;
    uint32_t out[2] = {0u, 0u};
    const uint64_t inv2 = b200::f2_pack(inv, inv), plus = b200::f2_pack(192.f, 192.f), minus = b200::f2_pack(-192.f, -192.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      b200::f2_unpack(b200::f2_add(b200::f2_fma(b200::f2_pack(v[2 * k], v[2 * k + 1]), inv2, plus), minus), a, b);
      out[k >> 2] |= e2m1x2_from_f32(copysignf(a, v[2 * k]), copysignf(b, v[2 * k + 1])) << (8 * (k & 3));
    }
    if (nan) out[0] = out[1] = 0u;
    *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * (D / 2)) = make_uint2(out[0], out[1]);
    sf[static_cast<size_t>(row) * LPR] = static_cast<uint8_t>(nan ? 0x7Fu : byte);
  }
}

// Reads positions back: a thread takes 8 values (4 bytes of codes, one 16-byte store) of each of its rows.
template <int D, bool F16>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_sm100(const __grid_constant__ Kv4MoveParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, U = kKv4WarpRows / RPP;
  const int which = blockIdx.y, lane = threadIdx.x & 31, unit = lane % LPR;
  const float up = f32_exp2i(which == 0 ? p.c.exp[0] : p.c.exp[1]);
  kv4_grid_wait();
  const Kv4MoveTile tile(p);
  const int r0 = (threadIdx.x >> 5) * kKv4WarpRows;
  const int start = p.first != nullptr ? kv4_clamp(p.first[tile.b], p.c.max_pages << p.c.page_shift) : 0;
  const int rows = kv4_len(p.c, tile.b) - start;     // rows that hold a position
  const int mine = tile.i0 + r0 + (lane & 7);
  const uint32_t my_row = kv4_lookup(p, tile.b, tile.h, lane < 8 && mine < rows && mine < p.N ? start + mine : -1);
  const uint8_t* const codes = (which == 0 ? p.c.codes[0] : p.c.codes[1]) + unit * 4;
  const uint8_t* const sf = (which == 0 ? p.c.sf[0] : p.c.sf[1]) + (unit >> 1);
  uint32_t w[U], byte[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t row = __shfl_sync(0xffffffffu, my_row, j * RPP + lane / LPR);
    w[j] = byte[j] = 0u;
    if (row != kNoRow) {
      w[j] = *reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(row) * (D / 2));
      byte[j] = sf[static_cast<size_t>(row) * (D / 16)];
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(which == 0 ? p.out[0] : p.out[1]) + tile.row0 * LPR + unit;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int r = r0 + j * RPP + lane / LPR;
    if (tile.i0 + r >= p.N) break;
    const uint32_t s2 = b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte[j] | (byte[j] << 8)));
    uint32_t f[4], out[4];
    f16x2_from_e2m1x8(w[j], f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = f32x2_from_f16x2(hmul2(f[k], s2));
      out[k] = pack_16<F16>(a.x * up, a.y * up);
    }
    dst[r * LPR] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace attn
