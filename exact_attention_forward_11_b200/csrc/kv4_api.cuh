// kv4_api.cuh - host side of include/kv4_b200.h (part of attn_api.cu: it uses that
// file's argument checks and launch helpers).
#pragma once

namespace {

// the int32 arrays may be slices of larger ones
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// whether two arrays of `bytes` bytes share any
bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x < y ? y - x : x - y) < bytes;
}

attn_status kv4_check_cache(const attn_kv4_cache* c, const int* block_table, const int* seq_lens, int B, int N,
                            int max_pages, int dtype) {
  if (c == nullptr || c->k_codes == nullptr || c->k_sf == nullptr || c->v_codes == nullptr || c->v_sf == nullptr ||
      block_table == nullptr || seq_lens == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (attn_status s = check_shape(B, c->Hkv, N); s != ATTN_OK) return s;
  if (c->num_pages < 1 || max_pages < 1 || c->page_size < 1) return ATTN_ERR_INVALID_ARG;
  if (c->k_exp < -32 || c->k_exp > 32 || c->v_exp < -32 || c->v_exp > 32) return ATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * c->page_size > (1ll << 30)) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(c->num_pages) * c->Hkv >= (1ll << 32) / c->page_size) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(c->k_codes) || !aligned16(c->k_sf) || !aligned16(c->v_codes) || !aligned16(c->v_sf) ||
      !aligned4(block_table) || !aligned4(seq_lens))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

attn::Kv4Cache kv4_cache_of(const attn_kv4_cache* from, const int* block_table, const int* seq_lens, int B, int max_pages) {
  attn::Kv4Cache c;
  c.codes[0] = static_cast<uint8_t*>(from->k_codes);
  c.codes[1] = static_cast<uint8_t*>(from->v_codes);
  c.sf[0] = static_cast<uint8_t*>(from->k_sf);
  c.sf[1] = static_cast<uint8_t*>(from->v_sf);
  c.block_table = block_table;
  c.seq_lens = seq_lens;
  c.B = B;
  c.H = from->Hkv;
  c.num_pages = from->num_pages;
  c.page_shift = __builtin_ctz(static_cast<unsigned>(from->page_size));
  c.max_pages = max_pages;
  c.exp[0] = from->k_exp;
  c.exp[1] = from->v_exp;
  return c;
}

// How attn_fwd_kv4 runs a shape (host only; it assumes the SMs of a B200, so that the
// workspace's size does not depend on the current device): by the query rows of one cached head.
struct Kv4Plan {
  int nt;                    // decode kernel: 8-row tiles per block; 0: the chunk kernel
  int row_blocks, ctas;
  bool fits;                 // the decode kernel's units (see Kv4Runs) stay below 2^31
  size_t ml_bytes, o_bytes, workspace;
};
constexpr int kKv4Sms = 148;
// The kernel, by the rows of a cached head and the work: the decode kernel in blocks of 8 (nt = 1) or 16 rows (2; a
// block reads the keys again, from L2), or the chunk kernel (0). Work is the units of Kv4Runs at the table's full
// length (the host does not know the sequences': a table with room counts as full), an item counting as its tiles and
// two. Both sides measured (8 cached heads unless said, d = 128 / d = 64, us):
//   * 9 to 16 and 25 to 32 rows: blocks of 16 (16 sequences of 4000 keys, d = 128: 16 rows 33.0, in blocks of 8 38.4; 32
//     rows 60 and 69). 17 to 24 rows: three blocks of 8 instead of two of 16 (54.7 and 59.1).
//   * above 32 rows: the chunk kernel (d = 128: 32 sequences of 8192 keys, 40 rows 219 and in the decode kernel 258; 8 of
//     6000 keys, 64 rows 60.6 and 76), but the decode kernel for up to 1600 units of 16 rows, where its start is the
//     shorter. Decode against chunk kernel: 864 units (48 rows, 6 x 1000 keys) 13.7 and 28.1 / 11.2 and 22.0; 1120 (100
//     rows, 2 x 2000) 18.5 and 28.1 / 15.3 and 21.4; 1536 (40 rows, 16 x 300) 22.7 and 27.0 / 18.0 and 21.2; 1680 (100 rows,
//     3 x 2000) 28.5 and 27.9 / 22.6 and 21.9; 1728 (48 rows, 12 x 1000) 25.0 and 34.9 / 18.3 and 26.6; 1920 (40 rows,
//     20 x 300) 29.1 and 28.8 / 22.8 and 22.4; 2240 (100 rows, 4 x 2000) 35.0 and 30.4 / 27.2 and 23.4.
//   * blocks of 8 for any rows up to 512 units of 8 rows. Blocks of 8 against 16: 320 units (32 rows, 2 x 700 keys) 9.4 and
//     11.3 / 8.1 and 9.3; 512 (64 rows, 2 x 500) 8.6 and 10.6 / 7.5 and 8.8; 640 (32 rows, 4 x 700) 12.2 and 11.5 / 9.6 and
//     9.7; 768 (16 rows, 8 x 1000) 14.4 and 13.4 / 11.1 and 10.9.
constexpr int kKv4DecodeRows = 32, kKv4DecodeUnits = 1600, kKv4SmallUnits = 512;

Kv4Plan kv4_plan(int B, int Hq, int Hkv, int N, int d, int page_size, int max_pages) {
  Kv4Plan r;
  const long long rows = static_cast<long long>(Hq / Hkv) * N;
  const long long positions = static_cast<long long>(max_pages) * page_size;
  auto work = [&](int block) {
    const double item = static_cast<double>((positions + attn::kDecTile - 1) / attn::kDecTile + attn::kDecSegmentTiles);
    return item * B * Hkv * static_cast<double>((rows + block - 1) / block);
  };
  if (rows <= 8 || (rows > 16 && rows <= 24) || work(8) <= kKv4SmallUnits)
    r.nt = 1;
  else
    r.nt = rows <= kKv4DecodeRows || work(16) <= kKv4DecodeUnits ? 2 : 0;
  const int block = r.nt > 0 ? 8 * r.nt : attn::kChunkRows, keys = r.nt > 0 ? attn::kDecTile : 128;
  r.row_blocks = static_cast<int>((rows + block - 1) / block);
  const long long tiles = (positions + keys - 1) / keys;
  const long long most = kKv4Sms * (r.nt == 1 ? 2 : 1);
  const double units = static_cast<double>(tiles) * B * Hkv * r.row_blocks;
  r.ctas = static_cast<int>(units < most ? units : most);
  r.fits = r.nt == 0 || work(block) < 2147483648.0;
  r.ml_bytes = static_cast<size_t>(2) * r.ctas * block * sizeof(float2);
  r.o_bytes = static_cast<size_t>(2) * r.ctas * block * d * sizeof(float);
  r.workspace = r.ml_bytes + r.o_bytes + (r.ctas * sizeof(attn::Kv4Head) + 15) / 16 * 16;
  return r;
}

// Launches a kernel that may start before the one before it in the stream has ended, and waits for it
// itself (kv4_grid_wait).
template <class P>
cudaError_t launch_after(void (*kern)(P), dim3 grid, int threads, int smem, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <class C, bool F16>
attn_status launch_kv4_dec(const attn::Kv4AttnParams& p, int tag, cudaStream_t stream) {
  auto kern = attn::kv4_decode_sm100<C, F16>;
  if (!set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, tag)) return ATTN_ERR_CUDA;
  cudaError_t e = launch_after(kern, dim3(p.ctas), attn::kDecWarps * 32, C::SMEM_BYTES, stream, p);
  if (e == cudaSuccess)
    e = launch_after(attn::kv4_join_sm100<C::D, C::ROWS, F16>, dim3(p.ctas, C::ROWS / 8), 256, 0, stream, p);
  if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) {
    forget_smem(tag);
    return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

template <int D, bool F16, bool PAIR>
attn_status launch_kv4_chunk(const attn::Kv4AttnParams& p, int tag, cudaStream_t stream, int fault_cta, uint64_t wait_limit) {
  using C = attn::Kv4ChunkCfg<D, PAIR>;
  auto kern = attn::kv4_chunk_sm100<C, F16>;
  if (!set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, tag)) return ATTN_ERR_CUDA;
  cudaError_t e = launch_after(kern, dim3(p.ctas), C::THREADS, C::SMEM_BYTES, stream,
                               attn::Kv4ChunkParams{p, wait_limit, fault_cta});
  if (e == cudaSuccess)
    e = launch_after(attn::kv4_join_sm100<D, attn::kChunkRows, F16>,
                     dim3(p.ctas, (PAIR ? 128 : attn::kChunkRows) / 8), 256, 0, stream, p);
  if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) {
    forget_smem(tag);
    return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

template <int D, bool F16>
attn_status launch_kv4_rows(const attn::Kv4AttnParams& p, const Kv4Plan& plan, cudaStream_t stream, int fault_cta,
                            uint64_t wait_limit) {
  const int tag = 16 + (D == 128 ? 0 : 8) + (F16 ? 4 : 0);
  if (plan.nt == 0)
    return p.Hq / p.c.H * p.N <= 128 ? launch_kv4_chunk<D, F16, true>(p, tag + 2, stream, fault_cta, wait_limit)
                                     : launch_kv4_chunk<D, F16, false>(p, tag + 3, stream, fault_cta, wait_limit);
  if (plan.nt == 1) return launch_kv4_dec<attn::Kv4DecCfg<D, 1>, F16>(p, tag, stream);
  return launch_kv4_dec<attn::Kv4DecCfg<D, 2>, F16>(p, tag + 1, stream);
}

}  // namespace

extern "C" {

attn_status attn_kv4_append(const attn_kv4_cache* cache, const void* k, const void* v, const int* block_table,
                            const int* seq_lens, const int* new_lens, int B, int N, int max_pages, attn_dtype dtype,
                            void* stream) {
  if (k == nullptr || v == nullptr) return ATTN_ERR_INVALID_ARG;
  if (attn_status s = kv4_check_cache(cache, block_table, seq_lens, B, N, max_pages, dtype); s != ATTN_OK) return s;
  if (!aligned16(k) || !aligned16(v) || !aligned4(new_lens)) return ATTN_ERR_MISALIGNED;
  attn::Kv4MoveParams p{};
  p.c = kv4_cache_of(cache, block_table, seq_lens, B, max_pages);
  p.in[0] = static_cast<const uint8_t*>(k);
  p.in[1] = static_cast<const uint8_t*>(v);
  p.first = new_lens;
  p.N = N;
  p.tiles = (N + attn::kKv4Rows - 1) / attn::kKv4Rows;
  const bool f16 = dtype == ATTN_FP16;
  auto kern = cache->d == 128 ? (f16 ? attn::kv4_append_sm100<128, true> : attn::kv4_append_sm100<128, false>)
                              : (f16 ? attn::kv4_append_sm100<64, true> : attn::kv4_append_sm100<64, false>);
  const cudaError_t e = launch_after(kern, dim3(static_cast<unsigned>(B * cache->Hkv * p.tiles), 2), attn::kKv4Threads, 0,
                                     static_cast<cudaStream_t>(stream), p);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_kv4_read(const attn_kv4_cache* cache, const int* block_table, const int* seq_lens, const int* starts,
                          void* k, void* v, int B, int N, int max_pages, attn_dtype dtype, void* stream) {
  if (k == nullptr || v == nullptr) return ATTN_ERR_INVALID_ARG;
  if (attn_status s = kv4_check_cache(cache, block_table, seq_lens, B, N, max_pages, dtype); s != ATTN_OK) return s;
  if (!aligned16(k) || !aligned16(v) || !aligned4(starts)) return ATTN_ERR_MISALIGNED;
  if (overlap(k, v, static_cast<size_t>(B) * cache->Hkv * N * cache->d * 2)) return ATTN_ERR_INVALID_ARG;
  attn::Kv4MoveParams p{};
  p.c = kv4_cache_of(cache, block_table, seq_lens, B, max_pages);
  p.out[0] = static_cast<uint8_t*>(k);
  p.out[1] = static_cast<uint8_t*>(v);
  p.first = starts;
  p.N = N;
  p.tiles = (N + attn::kKv4Rows - 1) / attn::kKv4Rows;
  const bool f16 = dtype == ATTN_FP16;
  auto kern = cache->d == 128 ? (f16 ? attn::kv4_read_sm100<128, true> : attn::kv4_read_sm100<128, false>)
                              : (f16 ? attn::kv4_read_sm100<64, true> : attn::kv4_read_sm100<64, false>);
  const cudaError_t e = launch_after(kern, dim3(static_cast<unsigned>(B * cache->Hkv * p.tiles), 2), attn::kKv4Threads, 0,
                                     static_cast<cudaStream_t>(stream), p);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_kv4_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int page_size, int max_pages) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0 || max_pages < 1) return 0;
  const Kv4Plan plan = kv4_plan(B, Hq, Hkv, N, d, page_size, max_pages);
  return plan.fits ? plan.workspace : 0;
}

}  // extern "C"

namespace {

attn_status fwd_kv4(const attn_kv4_cache* cache, const void* q, const int* block_table, const int* seq_lens,
                    const int* q_lens, void* o, float* lse, void* workspace, size_t workspace_bytes, int B, int Hq, int N,
                    int max_pages, float scale, int causal, attn_dtype dtype, void* stream, int fault_cta,
                    uint64_t wait_limit) {
  if (q == nullptr || o == nullptr || q == o || cache == nullptr) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  const int d = cache->d, Hkv = cache->Hkv;
  if (attn_status s = resolve_scale(scale, d > 0 ? d : 1); s != ATTN_OK) return s;
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (attn_status s = check_shape(B, Hq, N); s != ATTN_OK) return s;
  if (attn_status s = kv4_check_cache(cache, block_table, seq_lens, B, N, max_pages, dtype); s != ATTN_OK) return s;
  const Kv4Plan plan = kv4_plan(B, Hq, Hkv, N, d, cache->page_size, max_pages);
  if (!plan.fits || workspace == nullptr || workspace_bytes < plan.workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned4(q_lens) || !aligned16(workspace))
    return ATTN_ERR_MISALIGNED;
  if (overlap(q, o, static_cast<size_t>(B) * Hq * N * d * 2)) return ATTN_ERR_INVALID_ARG;
  attn::Kv4AttnParams p{};
  p.c = kv4_cache_of(cache, block_table, seq_lens, B, max_pages);
  p.q = static_cast<const uint8_t*>(q);
  p.o = static_cast<uint8_t*>(o);
  p.lse = lse;
  p.q_lens = q_lens;
  p.Hq = Hq;
  p.N = N;
  p.causal = causal;
  p.scale_log2 = std::ldexp(scale * 1.4426950408889634f, cache->k_exp);
  p.row_blocks = plan.row_blocks;
  p.ctas = plan.ctas;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + plan.ml_bytes);
  p.heads = reinterpret_cast<attn::Kv4Head*>(ws + plan.ml_bytes + plan.o_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = dtype == ATTN_FP16;
  if (d == 128)
    return f16 ? launch_kv4_rows<128, true>(p, plan, st, fault_cta, wait_limit)
               : launch_kv4_rows<128, false>(p, plan, st, fault_cta, wait_limit);
  return f16 ? launch_kv4_rows<64, true>(p, plan, st, fault_cta, wait_limit)
             : launch_kv4_rows<64, false>(p, plan, st, fault_cta, wait_limit);
}

}  // namespace

extern "C" {

attn_status attn_fwd_kv4(const attn_kv4_cache* cache, const void* q, const int* block_table, const int* seq_lens,
                         const int* q_lens, void* o, float* lse, void* workspace, size_t workspace_bytes, int B, int Hq,
                         int N, int max_pages, float scale, int causal, attn_dtype dtype, void* stream) {
  return fwd_kv4(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes, B, Hq, N, max_pages, scale,
                 causal, dtype, stream, -1, kWaitLimitCycles);
}

attn_status attn_fwd_kv4_inject_timeout(const attn_kv4_cache* cache, const void* q, const int* block_table,
                                        const int* seq_lens, const int* q_lens, void* o, float* lse, void* workspace,
                                        size_t workspace_bytes, int B, int Hq, int N, int max_pages, float scale,
                                        int causal, attn_dtype dtype, int fault_cta, unsigned long long wait_limit_cycles,
                                        void* stream) {
  if (fault_cta < 0 || wait_limit_cycles < 1024) return ATTN_ERR_INVALID_ARG;
  return fwd_kv4(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes, B, Hq, N, max_pages, scale,
                 causal, dtype, stream, fault_cta, wait_limit_cycles);
}

}  // extern "C"
