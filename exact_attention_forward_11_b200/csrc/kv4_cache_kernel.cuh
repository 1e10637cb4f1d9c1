// kv4_cache_kernel.cuh - the 4-bit key/value cache: its format on the device, and the
// kernels that quantise new tokens into it and read positions back
// (include/kv4_b200.h gives the definition).
//
// A row is one token of one head: d / 2 bytes of E2M1 codes and d / 16 E4M3 scale
// bytes. Both kernels move bytes and little else: a thread takes one block of 16
// values (32 bytes of 16-bit values, 8 bytes of codes, one scale byte), so a warp
// reads or writes 1 KB of consecutive values.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100.cuh"
#include "status.cuh"

namespace attn {

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

struct Kv4MoveParams {
  Kv4Cache c;
  const uint8_t* in[2];     // append: k, v [B, H, N, d] 16-bit values
  uint8_t* out[2];          // read: k, v
  const int* first;         // append: new_lens or nullptr; read: starts or nullptr
  int N;
  long long blocks;         // B * H * N * d / 16
};

// blockIdx.y: 0 keys, 1 values
template <int D, bool F16>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_sm100(const Kv4MoveParams p) {
  constexpr int BLK = D / 16;
  const int which = blockIdx.y;
  const float down = f32_exp2i(-p.c.exp[which]);
  for (long long t = static_cast<long long>(blockIdx.x) * kKv4Threads + threadIdx.x; t < p.blocks;
       t += static_cast<long long>(gridDim.x) * kKv4Threads) {
    const int blk = static_cast<int>(t % BLK);
    const uint32_t r = static_cast<uint32_t>(t / BLK);          // (b, h, i)
    const uint32_t bh = r / static_cast<uint32_t>(p.N);
    const int i = static_cast<int>(r - bh * p.N);
    const int b = static_cast<int>(bh / p.c.H), h = static_cast<int>(bh % p.c.H);
    const uint4* src = reinterpret_cast<const uint4*>(p.in[which] + t * 32);
    const uint4 x0 = src[0], x1 = src[1];
    const int n = p.first != nullptr ? kv4_clamp(p.first[b], p.N) : p.N;
    if (i >= n) continue;
    const int len = kv4_len(p.c, b);
    const int pos = len - n + i;
    if (pos < 0) {
      kv4_record(static_cast<unsigned long long>(static_cast<long long>(pos)));
      continue;
    }
    uint32_t row;
    if (!kv4_row(p.c, p.c.block_table[static_cast<long long>(b) * p.c.max_pages + (pos >> p.c.page_shift)], h, pos, row))
      continue;
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float v[16];
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = f32x2_from_16<F16>(w[k]);
      v[2 * k] = f.x * down;
      v[2 * k + 1] = f.y * down;
      amax = fmaxf(amax, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
      nan = nan || f.x != f.x || f.y != f.y;
    }
    const float want = fminf(fmaxf(__fdiv_rn(amax, 6.f), 0.001953125f), 448.f);
    const uint32_t byte = b200::pack_e4m3x4(want, 0.f, 0.f, 0.f) & 0xFFu;
    const float s = f32x2_from_f16x2(b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte))).x;
    uint32_t out[2] = {0u, 0u};
    if (!nan) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        out[k >> 2] |= e2m1x2_from_f32(__fdiv_rn(v[2 * k], s), __fdiv_rn(v[2 * k + 1], s)) << (8 * (k & 3));
    }
    *reinterpret_cast<uint2*>(p.c.codes[which] + static_cast<size_t>(row) * (D / 2) + blk * 8) =
        make_uint2(out[0], out[1]);
    p.c.sf[which][static_cast<size_t>(row) * BLK + blk] = static_cast<uint8_t>(nan ? 0x7Fu : byte);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_sm100(const Kv4MoveParams p) {
  constexpr int BLK = D / 16;
  const int which = blockIdx.y;
  const float up = f32_exp2i(p.c.exp[which]);
  for (long long t = static_cast<long long>(blockIdx.x) * kKv4Threads + threadIdx.x; t < p.blocks;
       t += static_cast<long long>(gridDim.x) * kKv4Threads) {
    const int blk = static_cast<int>(t % BLK);
    const uint32_t r = static_cast<uint32_t>(t / BLK);          // (b, h, i)
    const uint32_t bh = r / static_cast<uint32_t>(p.N);
    const int i = static_cast<int>(r - bh * p.N);
    const int b = static_cast<int>(bh / p.c.H), h = static_cast<int>(bh % p.c.H);
    const int start = p.first != nullptr ? kv4_clamp(p.first[b], p.c.max_pages << p.c.page_shift) : 0;
    const int len = kv4_len(p.c, b);
    uint32_t out[8] = {};
    uint32_t row;
    if (i < len - start &&
        kv4_row(p.c, p.c.block_table[static_cast<long long>(b) * p.c.max_pages + ((start + i) >> p.c.page_shift)], h,
                start + i, row)) {
      const uint2 w = *reinterpret_cast<const uint2*>(p.c.codes[which] + static_cast<size_t>(row) * (D / 2) + blk * 8);
      const uint32_t byte = p.c.sf[which][static_cast<size_t>(row) * BLK + blk];
      const uint32_t s2 = b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte | (byte << 8)));
      uint32_t f[4], g[4];
      f16x2_from_e2m1x8(w.x, f);
      f16x2_from_e2m1x8(w.y, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = f32x2_from_f16x2(hmul2(f[k], s2)), c = f32x2_from_f16x2(hmul2(g[k], s2));
        out[k] = pack_16<F16>(a.x * up, a.y * up);
        out[4 + k] = pack_16<F16>(c.x * up, c.y * up);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(p.out[which] + t * 32);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

}  // namespace attn
