// Definitions shared by the kernels of the 8-bit K/V tile cache: its geometry
// as the kernels take it, which tokens a call covers and which tiles a query
// can see.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <utility>

#include "veda_internal.cuh"

#define VEDA_KV_MAX_NB 8192  // table entries per (sequence, K/V head)

namespace veda {

struct KvGeom {
  int32_t B, hkv, d, tile, n_slots, nb_cap;
  uint8_t* k8;     // [n_slots, tile, d] e4m3
  uint8_t* v8;
  int32_t* table;  // [B, hkv, nb_cap]
  int32_t* pos;
  float* k_scale;
  float* v_scale;
  float* weight;
  int32_t* len;       // [B, hkv]
  int32_t* next_pos;  // [B]
  int32_t* arrive;    // [B, hkv], 0 between calls
  int32_t* dev_status;
};

// What the tail tiles were before pending tokens raised their scales (veda_kv_tail); codes NULL: not kept.
struct KvTail {
  uint8_t* codes;  // [B, hkv, 2 (K, V), tile, d]
  int4* key;       // [B, hkv, 2]: rows (0: nothing kept), slot, next_pos
  float2* scale;   // [B, hkv, 2]: before, raised
};

// bf16 rows [B, n, heads, d] with element strides (the last dimension is contiguous).
struct KvRows {
  const __nv_bfloat16* p;
  int64_t sb, sn, sh;
};

struct KvAttnParams {
  KvRows q;
  __nv_bfloat16* o;
  int64_t o_sb, o_sn, o_sh;
  int32_t heads, group, n_q;
  const int32_t* n_new;
  int32_t pending, causal, window, sinks, fill;
  float scale_log2;
  float* lse;     // [B, heads, n_q] natural log, or NULL
  float* weight;  // [B, hkv, nb_cap] or NULL
  float decay;
  // workspace, and how the rows (n_q * group per K/V head) are cut
  int32_t tiles;       // 1: the tile kernel (256 rows per CTA), 0: the row kernel
  int32_t alt;         // the tile kernel's B takes every second step of A's rows
  int32_t splits, parts, row_tiles, rows_cap, rows_pad, tile_rows;  // parts: of a row, for the join
  int32_t weight_blocks, join_rounds;  // blocks of a head that sum weights, and row groups of those behind, which join
  int32_t piece, pieces_cap;  // keys per entry of lw, entries per head
  float* part_o;   // [B, hkv, parts, rows_pad, d]
  int32_t* arrive;
  float2* part_ml; // [B, hkv, parts, rows_pad]: reference (log2) and sum
  float* lse2;     // [B, hkv, rows_cap] log2
  float* lw;       // [B, hkv, pieces_cap, rows_cap] log2 of a piece's sum
};

// New tokens of sequence b (n_new == NULL: all n), and the tokens its head h
// then holds; false, with VEDA_ERR_BAD_INDEX recorded, where the counts of the
// sequence are outside what the call or the cache can hold, for any of its heads:
// they share their positions, so one that stayed behind would read its later
// tokens at wrong ones. Every kernel of a step decides by this, so a sequence that
// is skipped is skipped by all of them. Called by whole warps.
__device__ __forceinline__ bool kv_counts(const KvGeom& g, int b, int h, int n, const int32_t* n_new, bool pending,
                                          int& n_b, int& held, int& total) {
  const int32_t* len = g.len + (long long)b * g.hkv;
  int most = 0, least = 0;  // over the heads, before n_new is waited for
#pragma unroll
  for (int x = 0; x < VEDA_MAX_HEADS; x += 32)
    if (x + threadIdx.x % 32 < g.hkv) {
      const int y = len[x + threadIdx.x % 32];
      most = max(most, y);
      least = min(least, y);
    }
  held = len[h];
  n_b = n_new ? n_new[b] : n;
  const bool bad = __any_sync(0xffffffffu, n_b < 0 || n_b > n || least < 0 ||
                                               (long long)most + (pending ? n_b : 0) > (long long)g.nb_cap * g.tile);
  if (bad) report(g.dev_status, VEDA_ERR_BAD_INDEX);
  total = held + (pending && !bad ? n_b : 0);
  return !bad;
}

// Whether any query at a position in [t_lo, t_hi] sees any token of a tile
// that starts at position p. Sums in 64 bits: positions may be near the ends
// of the range.
__device__ __forceinline__ bool kv_tile_seen(int p, int tile, int t_lo, int t_hi, int causal, int window, int sinks) {
  if (causal && p > t_hi) return false;
  return window <= 0 || p < sinks || (long long)p + tile - 1 > (long long)t_lo - window;
}

// A pool as a 2D map of bytes [rows, d], box [box_rows, d], swizzled over d bytes (64 or 128).
CUresult encode_tensor_map_2d_u8(CUtensorMap* map, const void* base, uint64_t d, uint64_t rows, uint32_t box_rows);

// The kernels are launched so that each may be
// set up while the one before it in the stream ends: it waits here for that one's
// results, before it reads or writes anything, and lets the next one do the same.
__device__ __forceinline__ void after_predecessor() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, Args&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Lets a kernel have `bytes` of dynamic shared memory, once per device: `done`,
// a bit per device, is the caller's own for this kernel.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_kv_append(const KvGeom& g, const KvTail& tail, const KvRows& k, const KvRows& v, int n,
                             const int32_t* n_new, cudaStream_t s);
cudaError_t launch_kv_advance(const KvGeom& g, int n, const int32_t* n_new, cudaStream_t s);
cudaError_t launch_kv_evict(const KvGeom& g, const int32_t* keep, int sink, int recent, const KvGeom& out,
                            cudaStream_t s);
size_t kv_attn_ws_bytes(const KvGeom& g, int heads, int n_q, bool weights);
cudaError_t launch_kv_attn(const KvGeom& g, KvAttnParams p, void* ws, cudaStream_t s);
// workspace of the call, and its pointers and split into the parameters
size_t kv_attn_plan(const KvGeom& g, KvAttnParams& p, bool weights, uint8_t* ws);

}  // namespace veda
