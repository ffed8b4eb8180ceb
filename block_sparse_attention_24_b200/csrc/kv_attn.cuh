// Device code that both attention kernels of the 8-bit K/V tile cache use.
#pragma once

#include "kv_internal.cuh"

namespace veda {

// The two code pools as [n_slots * tile, d] bytes.
struct KvMaps {
  CUtensorMap k, v;
};

constexpr float OFF = 7.f;  // see kv_attn.cu
constexpr float LN2 = 0.69314718055994531f;

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// two f16 pairs from four e4m3 codes
__device__ __forceinline__ void codes_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The larger magnitude of two bf16 values, as fp32 bits (infinities and NaN
// above every finite value).
__device__ __forceinline__ uint32_t bf16x2_top(uint32_t w) { return max((w << 16) & 0x7fffffffu, w & 0x7fff0000u); }

// Four bf16 values times `mul` as two e4m3 parts each: the nearest code, and
// the nearest to what it leaves.
__device__ __forceinline__ void split_e4m3x4(uint32_t w0, uint32_t w1, float mul, uint32_t& hi, uint32_t& lo) {
  const float x[4] = {__uint_as_float(w0 << 16) * mul, __uint_as_float(w0 & 0xffff0000u) * mul,
                      __uint_as_float(w1 << 16) * mul, __uint_as_float(w1 & 0xffff0000u) * mul};
  hi = pack_e4m3x4(x[0], x[1], x[2], x[3]);
  uint32_t a, b;
  codes_f16(hi, a, b);
  const float2 y = __half22float2(*reinterpret_cast<__half2*>(&a)), z = __half22float2(*reinterpret_cast<__half2*>(&b));
  lo = pack_e4m3x4(x[0] - y.x, x[1] - y.y, x[2] - z.x, x[3] - z.y);
}

// The power of two that takes a row whose largest |value| has the bits `top`
// into [2^E, 2^(E+1)), and its inverse, which is NaN for a row that is not
// finite (and so are its logits then).
template <int E>
__device__ __forceinline__ void q_scale(uint32_t top, float& mul, float& inv) {
  int ex = 127 + E - ((int)(top >> 23) - 127);
  if (ex > 253) ex = 253;
  if (ex < 1) ex = 1;
  mul = __uint_as_float((uint32_t)ex << 23);
  inv = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(254 - ex) << 23);
}

// 16-byte chunk `ch` of row r of D-byte rows in shared memory: chunks are
// permuted inside each 128 bytes so that eight rows' chunks fall into
// different banks (TMA's and tcgen05's 128- and 64-byte swizzles).
template <int D>
__device__ __forceinline__ int code_at(int r, int ch) {
  return D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}

// The tiles that queries at positions t_lo .. t_hi see: entries [0, n_first)
// and [from, upto) of the table. Counted by the whole block from the
// positions, which ascend, and only where the mask may hide some; `last_t` is
// the position of the sequence's last query, `cnt` zeroed shared memory.
struct KvRange {
  int n_first, from, upto;
  __device__ int count() const { return n_first + upto - from; }
  __device__ int tile(int vt) const { return vt < n_first ? vt : vt - n_first + from; }
};
__device__ __forceinline__ KvRange kv_range(const KvGeom& g, const KvAttnParams& p, long long trow, int nb, int t_lo,
                                            int t_hi, int last_t, int* cnt, int tid, int threads) {
  KvRange r{0, 0, nb};
  if (p.window > 0 || (p.causal && t_hi < last_t)) {
    int a = 0, f = 0, u = 0;
    for (int i = tid; i < nb; i += threads) {
      const int ps = g.pos[trow + i];
      const bool ahead = p.causal && ps > t_hi;
      u += !ahead;
      if (p.window > 0 && !ahead) {
        a += ps < p.sinks;
        f += (long long)ps + g.tile - 1 <= (long long)t_lo - p.window;
      }
    }
    a = __reduce_add_sync(0xffffffffu, a);
    f = __reduce_add_sync(0xffffffffu, f);
    u = __reduce_add_sync(0xffffffffu, u);
    if (tid % 32 == 0) {
      atomicAdd(&cnt[0], a);
      atomicAdd(&cnt[1], f);
      atomicAdd(&cnt[2], u);
    }
    __syncthreads();
    r.upto = cnt[2];
    r.from = cnt[1];
    r.n_first = min(cnt[0], r.from);
  }
  return r;
}

cudaError_t launch_kv_attn_tiles(const KvGeom& g, const KvAttnParams& p, cudaStream_t s);

}  // namespace veda
