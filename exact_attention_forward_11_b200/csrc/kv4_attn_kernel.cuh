// kv4_attn_kernel.cuh - attention over the 4-bit cache (include/kv4_b200.h).
//
// One CTA of 128 threads per query row, two passes over each tile of 128 keys: a thread
// scores one key (fp32), then a thread owns one output channel and sums the tile's
// P V. Online softmax over the tiles.
#pragma once

#include "kv4_cache_kernel.cuh"

namespace attn {

struct Kv4AttnParams {
  Kv4Cache c;
  const uint8_t* q;          // [B, Hq, N, d]
  uint8_t* o;
  float* lse;                // or nullptr
  const int* q_lens;         // or nullptr
  int Hq, N, causal;
  float scale_log2;          // scale * log2(e) * 2^k_exp
};

template <int D, bool F16>
__global__ void __launch_bounds__(128) kv4_attn_row_sm100(const Kv4AttnParams p) {
  __shared__ float qs[D], ps[128], red[4];
  __shared__ uint32_t rows[128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x % p.N, hq = (blockIdx.x / p.N) % p.Hq, b = blockIdx.x / p.N / p.Hq;
  const int h = hq / (p.Hq / p.c.H);
  const int n = p.q_lens != nullptr ? kv4_clamp(p.q_lens[b], p.N) : p.N;
  if (i >= n) return;
  const int len = kv4_len(p.c, b);
  const int end = p.causal ? min(len, len - n + i + 1) : len;
  const size_t r = blockIdx.x;
  if (tid < D / 2) {
    const float2 f = f32x2_from_16<F16>(reinterpret_cast<const uint32_t*>(p.q + r * D * 2)[tid]);
    qs[2 * tid] = f.x;
    qs[2 * tid + 1] = f.y;
  }
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 < end; j0 += 128) {
    __syncthreads();
    const int j = j0 + tid;
    float s = -INFINITY;
    uint32_t row = 0xFFFFFFFFu;
    if (j < end && kv4_row(p.c, p.c.block_table[static_cast<long long>(b) * p.c.max_pages + (j >> p.c.page_shift)], h, j, row)) {
      s = 0.f;
      for (int blk = 0; blk < D / 16; ++blk) {
        const uint2 w = *reinterpret_cast<const uint2*>(p.c.codes[0] + static_cast<size_t>(row) * (D / 2) + blk * 8);
        const uint32_t byte = p.c.sf[0][static_cast<size_t>(row) * (D / 16) + blk];
        const uint32_t s2 = b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte | (byte << 8)));
        uint32_t f[4], g[4];
        f16x2_from_e2m1x8(w.x, f);
        f16x2_from_e2m1x8(w.y, g);
        for (int k = 0; k < 4; ++k) {
          const float2 a = f32x2_from_f16x2(hmul2(f[k], s2)), c = f32x2_from_f16x2(hmul2(g[k], s2));
          s += a.x * qs[blk * 16 + 2 * k] + a.y * qs[blk * 16 + 2 * k + 1] + c.x * qs[blk * 16 + 8 + 2 * k] +
               c.y * qs[blk * 16 + 9 + 2 * k];
        }
      }
      s *= p.scale_log2;
    } else {
      row = 0xFFFFFFFFu;
    }
    rows[tid] = row;
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float pj = exp2f(s - m_use);
    ps[tid] = pj;
    float sum = pj;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    const float alpha = exp2f(m - m_use);
    l = l * alpha + (red[0] + red[1] + red[2] + red[3]);
    m = m_new;
    acc *= alpha;
    if (tid < D) {
      const int kn = min(128, end - j0);
      for (int k = 0; k < kn; ++k) {
        const uint32_t rk = rows[k];
        if (rk == 0xFFFFFFFFu) continue;
        const uint32_t cb = reinterpret_cast<const uint32_t*>(p.c.codes[1] + static_cast<size_t>(rk) * (D / 2))[tid >> 3];
        const uint32_t byte = p.c.sf[1][static_cast<size_t>(rk) * (D / 16) + (tid >> 4)];
        uint32_t f[4];
        f16x2_from_e2m1x8(cb, f);
        const float2 a = f32x2_from_f16x2(hmul2(f[(tid >> 1) & 3], b200::f16x2_from_e4m3x2(static_cast<uint16_t>(byte | (byte << 8)))));
        acc += ps[k] * ((tid & 1) ? a.y : a.x);
      }
    }
  }
  if (tid < D) {
    const float o = l > 0.f || l != l ? acc / l * f32_exp2i(p.c.exp[1]) : 0.f;
    reinterpret_cast<uint16_t*>(p.o)[r * D + tid] = static_cast<uint16_t>(pack_16<F16>(o, 0.f));
  }
  if (p.lse != nullptr && tid == 0) p.lse[r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace attn
