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
// Whether the phase of `bar` with this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
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
// and [from, upto) of the table. Counted by `threads` threads that `sync` joins
// from the positions, which ascend, and only where the mask may hide some;
// `last_t` is the position of the sequence's last query, `cnt` zeroed shared
// memory.
struct KvRange {
  int n_first, from, upto;
  __device__ int count() const { return n_first + upto - from; }
  __device__ int tile(int vt) const { return vt < n_first ? vt : vt - n_first + from; }
};
template <class Sync>
__device__ __forceinline__ KvRange kv_range(const KvGeom& g, const KvAttnParams& p, long long trow, int nb, int t_lo,
                                            int t_hi, int last_t, int* cnt, int tid, int threads, Sync sync) {
  KvRange r{0, 0, nb};
  if (p.window > 0 || (p.causal && t_hi < last_t)) {
    int a = 0, f = 0, u = 0;
#pragma unroll 4
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
    sync();
    r.upto = cnt[2];
    r.from = cnt[1];
    r.n_first = min(cnt[0], r.from);
  }
  return r;
}

// Zeros, and lse = -inf, for the rows of a head that no query is in (p.fill):
// rows lo .. hi-1, by `threads` threads. Not inlined, as the kernels' registers
// then go to it too (32 x 2 tokens of 16 rows, window 2,048: 20.2 us, not 19.7).
template <int D>
__device__ __noinline__ void fill_rows_at(__nv_bfloat16* o, long long sn, long long sh, float* lse, int n_q, int group,
                                          int lo, int hi, int x0, int threads) {
#pragma unroll 1
  for (long long x = (long long)lo * (D / 8) + x0; x < (long long)hi * (D / 8); x += threads) {
    const int r = (int)(x / (D / 8)), c8 = (int)(x % (D / 8)), i = r / group, y = r - i * group;
    *reinterpret_cast<uint4*>(o + i * sn + y * sh + c8 * 8) = make_uint4(0, 0, 0, 0);
    if (c8 == 0 && lse) lse[(long long)y * n_q + i] = -INFINITY;
  }
}
template <int D>
__device__ __forceinline__ void fill_rows(const KvAttnParams& p, int b, int h, int lo, int hi, int tid, int threads) {
  const int qh = h * p.group;
  fill_rows_at<D>(p.o + b * p.o_sb + qh * p.o_sh, p.o_sn, p.o_sh,
                  p.lse ? p.lse + ((long long)b * p.heads + qh) * p.n_q : nullptr, p.n_q, p.group, lo, hi, tid, threads);
}

// ------------------------------------------------------- steps of 128 keys
constexpr int STEP = 128, HALF = 64;  // a step is two halves of 64 keys, each a TMA box of its own

// What a step's consumers need to know. Written before the step's copies are
// announced, so whoever has seen those copies (or an MMA on them) complete can
// read it.
struct StepMeta {
  float ks[2], ev[2], rv[2];  // K scale, log2 of the V scale, its inverse
  int pos[2], left[2];        // first position, keys that exist
  int entry[2];               // table entry, -1 for none
  int full;                   // every query of the CTA sees all 128 keys
  int pad;
};
static_assert(sizeof(StepMeta) % 8 == 0, "barriers follow");

// The producer warp's view of the steps: lane j holds what half j of the next
// 16 steps needs, so a step's table entry and scales cost no latency.
struct StepFeed {
  int pool, entry, pos, left;
  float ks, vs;

  // halves of steps e .. e+15 of this CTA, whose first step is s_lo of all
  __device__ void load(const KvGeom& g, long long trow, const KvRange& rg, int total, int s_lo, int e, int n_steps,
                       int lane) {
    const int half = 2 * (s_lo + e) + lane, one = g.tile == STEP;  // 64-key halves of the tiles seen
    const int vt = one ? half >> 1 : half, sub = one ? half & 1 : 0;
    pool = entry = -1;
    pos = left = 0;
    ks = 0.f;
    vs = 1.f;
    if (vt < rg.count() && e + (lane >> 1) < n_steps) {
      const int i = rg.tile(vt);
      const int slot = g.table[trow + i];
      entry = i;
      pos = g.pos[trow + i] + sub * HALF;
      const float k = g.k_scale[trow + i], v = g.v_scale[trow + i];
      if (slot >= 0 && slot < g.n_slots) {
        left = max(0, min(HALF, total - (i * g.tile + sub * HALF)));
        pool = left > 0 ? slot * g.tile + sub * HALF : -1;
        ks = k;
        vs = v;
      } else {
        report(g.dev_status, VEDA_ERR_BAD_INDEX);
      }
    }
  }

  // The description of step e (all lanes call), and the pool rows of its
  // halves (-1: no copy).
  __device__ void put(StepMeta& m, const KvGeom& g, const KvAttnParams& p, int e, int t_lo, int t_hi, int lane,
                      int& row0, int& row1) const {
    const int l0 = 2 * (e & 15);
    const bool seen = left == HALF && (!p.causal || pos + HALF - 1 <= t_lo) &&
                      (p.window <= 0 || pos + HALF <= p.sinks || (long long)pos > (long long)t_hi - p.window);
    const int both = (__ballot_sync(0xffffffffu, seen) >> l0 & 3u) == 3u;
    if (lane == l0 || lane == l0 + 1) {
      const int x = lane & 1;
      m.ks[x] = ks;
      m.ev[x] = log2f(vs);
      m.rv[x] = 1.0f / vs;
      m.pos[x] = pos;
      m.left[x] = left;
      m.entry[x] = entry;
      m.full = both;
    }
    row0 = __shfl_sync(0xffffffffu, pool, l0);
    row1 = __shfl_sync(0xffffffffu, pool, l0 + 1);
  }
};

// D[tmem] (+)= A * B on e4m3 operands in shared memory.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc),
      "r"(acc) : "memory");
}
// Instruction descriptor for M x N with fp32 D and A, B of format 0 (e4m3, or fp16 in kind::f16).
__host__ __device__ constexpr uint32_t idesc_fmt0(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Operand of D-byte rows in shared memory, swizzled over them (128 or 64
// bytes), eight rows to an atom; `lbo`: bytes between column groups where the
// rows run along K.
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(uint32_t saddr, uint32_t lbo = 16) {
  uint64_t d = sdesc_sw128(saddr, lbo, 8 * D);
  if (D == 64) d = (d & ~((uint64_t)7 << 61)) | ((uint64_t)4 << 61);  // SWIZZLE_64B
  return d;
}

cudaError_t launch_kv_attn_tiles(const KvGeom& g, const KvAttnParams& p, cudaStream_t s);

}  // namespace veda
