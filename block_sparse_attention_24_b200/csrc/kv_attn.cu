// Attention over the 8-bit K/V tile cache: the plan of a call, the kernel for
// few query rows per K/V head (single tokens and their groups), and what joins
// the parts of the other one (kv_tiles.cu).
//
// Row r of a K/V head is query token r / group, query head h*group + r % group.
// With c the codes, s the tile scales and x_ij = scale*log2(e) * (q_i . ck_j)
// * sk + log2(sv):
//   P_ij = 2^(x_ij - M_i + OFF),  O_i = sum_j P_ij cv_j / sum_j P_ij / sv.
// The V scale is part of the exponent, so P V runs on the bare codes and tiles
// of any scale add up in one accumulator; dividing P by sv again for the sum is
// exact for powers of two. M is a reference, not the maximum: it moves only
// when some x passes it by a margin, so that P stays within its type (fp16 in
// the tile kernel, e4m3 parts here). Sums, references and O are fp32.
#include <climits>
#include <cmath>

#include "kv_attn.cuh"

namespace veda {
namespace {

// Few rows: HBM is the bound (1 byte per K and V value, each used by up to 16
// rows), so the codes go from TMA straight into tcgen05 MMAs on e4m3 and no
// thread touches them; converting them first (mma.sync on fp16) took 840
// instructions per 32 keys and ran at 4.1 TB/s.
//   S^T = K Q^T   A = the K tile (128 keys x d), B = Q: each row, times a power
//                 of two, in four e4m3 parts of which each holds 16 times what
//                 the one before left, N = 4 RP columns; a row's logit is the
//                 sum of its four columns with weights 16^-k.
//   O^T = V^T P   A = the V tile taken along its rows (d x 128 keys; for d = 64
//                 the upper half of M repeats the lower), B = P^T, in four
//                 parts too: 16 bits, down to 2^-29 of the row's largest.
// A thread owns a key (TMEM lane) of S^T and a channel of O^T, for four or
// eight rows; the rows are columns, so the work per key goes with the rows there
// are, and from five rows on two warpgroups share it. S and P are
// double-buffered: a step's S is issued as soon as its K has arrived, beside
// the softmax of the step before.
//   warps 0-3 (0-7)  softmax
//   then one warp    producer: table, scales, TMA
//   and one          MMA issuer (one thread; issuing blocks it, so it is no
//                    softmax thread)
// The CTAs that share a head's keys count themselves in `arrive`; the last one
// joins their parts, and sums the tile weights.
// Measured: 2 sequences x 24 heads x 80,640 keys, d = 128: 155 us, 6.4 TB/s (98%
// of a measured copy); 16 sequences of up to 8,190 keys, 32/8 heads, with
// weights: 46 us, 4.4 TB/s; 1,500 keys, 32/8 heads: 9.5 us, a chain of latencies.
// A head's CTAs as a cluster that exchanges its parts through shared memory took
// the same (1,500 keys) or more (window 2,048: 27 against 22 us; 80,640 keys: 223
// against 154 us): clusters leave SM slots empty.
// Up to 16 rows: at 32 rows and 16 x 8,190 keys two passes of this kernel would
// take 170 us, the tile kernel takes 93.
constexpr int FEW_ROWS = 16;
constexpr float MARGIN = 1.5f;  // P <= 2^(OFF + MARGIN) = 362 < 448

template <int D, int RP>
struct RowsCfg {
  static constexpr int N = 4 * RP;
  static constexpr int G = RP == 4 ? 1 : 2, R = RP / G;         // softmax warpgroups, rows of a thread
  static constexpr int SM = 128 * G, THREADS = SM + 64;
  static constexpr int CB = STEP * D;                           // bytes of a step's K or V codes
  static constexpr int ST = D == 64 ? (RP == 16 ? 5 : 6) : (RP == 16 ? 2 : 3);  // ring stages: two CTAs per SM
  static constexpr int OFF_Q = ST * 2 * CB;
  static constexpr int OFF_P = OFF_Q + N * D;
  static constexpr int OFF_META = OFF_P + 2 * N * STEP;
  static constexpr int OFF_BAR = OFF_META + ST * (int)sizeof(StepMeta);
  static constexpr int NUM_BARS = 3 * ST + 5;                   // K, V, free per stage; S, P twice; drain
  // float [4][RP], then [RP] factors, int [2][RP] position bounds
  static constexpr int OFF_RED = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_MISC = OFF_RED + 7 * RP * 4;
  static constexpr int ALLOC = OFF_MISC + 32 + 1024;
  static constexpr int TMEM = 4 * N;                            // S^T twice, O^T
  static_assert(2 * (ALLOC + 1024) <= 233472, "two CTAs per SM");
};

template <int SM>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(SM) : "memory");
}
template <int SM>
__device__ __forceinline__ bool softmax_any(bool x) {
  int r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((int)x), "n"(SM) : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&u)[N]) {
  if constexpr (N == 16) tmem_ld16(addr, u);
  else tmem_ld32(addr, u);
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&u)[N]) {
  if constexpr (N == 16) tmem_st16(addr, u);
  else tmem_st32(addr, u);
}

// Sums of every row's value over the warp, the rows halved between the lanes
// at each step: v[0] of the lanes from r * (32 / RP) on is row r's sum, and
// ref[0] the row's `ref`.
template <int N, int DIST, int RP>
__device__ __forceinline__ void warp_rows(float (&v)[RP], float (&ref)[RP], int lane) {
  if constexpr (N > 1) {
    const bool up = lane & DIST;
#pragma unroll
    for (int r = 0; r < N / 2; ++r) {
      const float keep = up ? v[N / 2 + r] : v[r], give = up ? v[r] : v[N / 2 + r];
      v[r] = keep + __shfl_xor_sync(0xffffffffu, give, DIST);
      ref[r] = up ? ref[N / 2 + r] : ref[r];
    }
    warp_rows<N / 2, DIST / 2>(v, ref, lane);
  } else {
#pragma unroll
    for (int d = DIST; d; d /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
  }
}

// Two values as four e4m3 parts each: part k is the code nearest to 16 times
// what part k-1 left. The codes of x are in the low bytes, those of y above.
__device__ __forceinline__ void four_parts(float x, float y, uint16_t (&c)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[k]) : "f"(y), "f"(x));
    if (k < 3) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c[k]));
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
      x = (x - f.x) * 16.f;
      y = (y - f.y) * 16.f;
    }
  }
}

template <int D, int RP>
__global__ void __launch_bounds__((RowsCfg<D, RP>::THREADS), 2)
    kv_attn_rows_kernel(const KvGeom g, const KvAttnParams p, const __grid_constant__ KvMaps maps) {
  using Cfg = RowsCfg<D, RP>;
  constexpr int N = Cfg::N, ST = Cfg::ST, R = Cfg::R, SM = Cfg::SM, THREADS = Cfg::THREADS;
  constexpr int PRODUCER = SM / 32, ISSUER = PRODUCER + 1;  // warps
  // column of part k of a row: a warpgroup's rows are side by side
  auto column = [](int k, int r) { return r / R * (4 * R) + k * R + r % R; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  const int sp = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  after_predecessor();
  int n_b, held, total;
  const int t_lo = g.next_pos[b];
  const bool fits = kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total);
  const int rows = fits ? n_b * p.group : 0;
  if (p.fill && sp == 0) fill_rows<D>(p, b, h, rows, p.rows_cap, tid, THREADS);
  if (rows == 0) return;
  const int bh = b * g.hkv + h;
  const long long trow = (long long)bh * g.nb_cap;
  const int t_hi = t_lo + n_b - 1;
  // Q: TPR threads per row
  constexpr int TPR = SM / RP, EL = D / TPR;
  const int qr = tid / TPR, qd = tid % TPR * EL;
  uint32_t qw[EL / 2];
#pragma unroll
  for (int x = 0; x < EL / 2; ++x) qw[x] = 0;
  if (qr < rows && warp < PRODUCER) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q.p + b * p.q.sb + (long long)(qr / p.group) * p.q.sn +
                                                            (long long)(h * p.group + qr % p.group) * p.q.sh + qd);
#pragma unroll
    for (int x = 0; x < EL / 2; ++x) qw[x] = src[x];
  }

  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* v_full = k_full + ST;
  uint64_t* free_ = v_full + ST;  // P V of the stage's step has completed
  uint64_t* s_full = free_ + ST;  // [2]
  // [2], an arrival per softmax thread each: with one, the softmax of the next step, whose S is
  // there already, could complete the phase after before this one is seen
  uint64_t* p_full = s_full + 2;
  uint64_t* drain = p_full + 2;
  StepMeta* meta = reinterpret_cast<StepMeta*>(smem + Cfg::OFF_META);
  float* red = reinterpret_cast<float*>(smem + Cfg::OFF_RED);
  float* qs = red + 4 * RP;
  int* seen_hi = reinterpret_cast<int*>(qs + RP);  // a row sees positions p <= hi && (p > lo || p < sinks)
  int* seen_lo = seen_hi + RP;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  int* cnt = reinterpret_cast<int*>(smem + Cfg::OFF_MISC + 8);  // [3], then a flag
  if (p.window > 0) {
    if (tid < 3) cnt[tid] = 0;
    __syncthreads();
  }
  const int nb = (total + g.tile - 1) / g.tile;
  const KvRange rg = kv_range(g, p, trow, nb, t_lo, t_hi, t_hi, cnt, tid, THREADS, [] { __syncthreads(); });
  const int per_step = STEP / g.tile;
  const int steps_all = (rg.count() + per_step - 1) / per_step;
  const int per = max(1, (steps_all + p.splits - 1) / p.splits);
  const int parts = max(1, (steps_all + per - 1) / per);  // CTAs that have steps (one, if there are none)
  if (sp >= parts) return;
  const int s_lo = sp * per, n_steps = max(0, min(per, steps_all - s_lo));

  // Each warp prepares its part before the one barrier: the first copies are
  // under way while Q is converted.
  StepFeed feed;
  int fed = 0;  // steps whose copies were issued (the producer's)
  auto produce = [&](int e) {
    if ((e & 15) == 0) feed.load(g, trow, rg, total, s_lo, e, n_steps, lane);
    const int st = e % ST;
    int row0, row1;
    feed.put(meta[st], g, p, e, t_lo, t_hi, lane, row0, row1);
    __syncwarp();
    if (lane == 0) {
      const uint32_t bytes = (row0 >= 0 ? Cfg::CB / 2 : 0) + (row1 >= 0 ? Cfg::CB / 2 : 0);
      uint8_t* kd = smem + st * 2 * Cfg::CB;
      uint8_t* vd = kd + Cfg::CB;
      mbar_expect_tx(k_full + st, bytes);
      if (row0 >= 0) tma_load_2d(kd, &maps.k, k_full + st, 0, row0);
      if (row1 >= 0) tma_load_2d(kd + Cfg::CB / 2, &maps.k, k_full + st, 0, row1);
      mbar_expect_tx(v_full + st, bytes);
      if (row0 >= 0) tma_load_2d(vd, &maps.v, v_full + st, 0, row0);
      if (row1 >= 0) tma_load_2d(vd + Cfg::CB / 2, &maps.v, v_full + st, 0, row1);
    }
    __syncwarp();
  };
  if (warp == PRODUCER) {
    if (lane < Cfg::NUM_BARS) mbar_init(k_full + lane, k_full + lane == p_full || k_full + lane == p_full + 1 ? SM : 1);
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    __syncwarp();
    for (; fed < ST && fed < n_steps; ++fed) produce(fed);
  } else if (warp == ISSUER) {
    tmem_alloc(tmem_slot, Cfg::TMEM);
    tmem_relinquish();
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int x = 0; x < EL / 2; ++x) top = max(top, bf16x2_top(qw[x]));
#pragma unroll
    for (int d = 1; d < TPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    float mul, inv;
    q_scale<7>(top, mul, inv);
    if (tid % TPR == 0) {
      qs[qr] = inv * p.scale_log2;
      const int t = t_lo + min(qr, rows - 1) / p.group;
      seen_hi[qr] = p.causal ? t : INT_MAX;
      seen_lo[qr] = p.window > 0 ? (int)max((long long)INT_MIN, (long long)t - p.window) : INT_MIN;
    }
#pragma unroll
    for (int x = 0; x < EL / 2; ++x) {
      uint16_t c[4];
      four_parts(__uint_as_float(qw[x] << 16) * mul, __uint_as_float(qw[x] & 0xffff0000u) * mul, c);
      const int d = qd + 2 * x;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint16_t*>(smem + Cfg::OFF_Q + code_at<D>(column(k, qr), d >> 4) + (d & 15)) = c[k];
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == PRODUCER) {
    // ------------------------------------------------------------- producer
    int e = fed;
    for (; e < n_steps; ++e) {
      if (!__all_sync(0xffffffffu, mbar_wait(free_ + e % ST, (e / ST - 1) & 1, abort_flag, g.dev_status))) break;
      produce(e);
    }
    if (*abort_flag && lane == 0)  // let every copy that was started land
      for (int x = max(0, e - ST); x < e; ++x) {
        mbar_wait_drain(k_full + x % ST, (x / ST) & 1, VEDA_WAIT_LIMIT_NS);
        mbar_wait_drain(v_full + x % ST, (x / ST) & 1, VEDA_WAIT_LIMIT_NS);
      }
  } else if (warp == ISSUER) {
    // ----------------------------------------------------------- MMA issuer
    if (lane == 0 && n_steps > 0) {
      constexpr uint32_t idesc_s = idesc_fmt0(128, N, false, false), idesc_o = idesc_fmt0(128, N, true, false);
      const uint64_t dK = sdesc_codes<D>(smem_u32(smem)), dV = sdesc_codes<D>(smem_u32(smem + Cfg::CB), 0);
      const uint64_t dQ = sdesc_codes<D>(smem_u32(smem + Cfg::OFF_Q)), dP = sdesc_codes<128>(smem_u32(smem + Cfg::OFF_P));
      auto issue_s = [&](int e) {  // its K has arrived, and P V of step e-2 has been issued
        const int st = e % ST;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          umma_f8_ss(tmem + (e & 1) * N, dK + (uint64_t)((st * 2 * Cfg::CB + kk * 32) >> 4), dQ + (uint64_t)(kk * 32 >> 4),
                     idesc_s, kk > 0);
        umma_commit(s_full + (e & 1));
      };
      auto k_here = [&](int e) { return mbar_wait(k_full + e % ST, (e / ST) & 1, abort_flag, g.dev_status); };
      bool ok = k_here(0);
      if (ok) issue_s(0);
      for (int e = 0; ok && e < n_steps; ++e) {
        const int st = e % ST;
        bool ahead = e + 1 == n_steps;  // S of the next step is issued
        // whichever comes first: the next K, or this P
        for (int spin = 0; spin < 4096 && !mbar_test(p_full + (e & 1), (e >> 1) & 1); ++spin)
          if (!ahead && mbar_test(k_full + (e + 1) % ST, ((e + 1) / ST) & 1)) {
            issue_s(e + 1);
            ahead = true;
          }
        ok = mbar_wait(p_full + (e & 1), (e >> 1) & 1, abort_flag, g.dev_status) &&
             mbar_wait(v_full + st, (e / ST) & 1, abort_flag, g.dev_status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < STEP / 32; ++q)
          umma_f8_ss(tmem + 2 * N, dV + (uint64_t)((st * 2 * Cfg::CB + q * 32 * D) >> 4),
                     dP + (uint64_t)(((e & 1) * N * STEP + q * 32) >> 4), idesc_o, (e > 0 || q > 0) ? 1u : 0u);
        umma_commit(free_ + st);
        if (!ahead) {
          ok = k_here(e + 1);
          if (ok) issue_s(e + 1);
        }
      }
      umma_commit(drain);
      mbar_wait_drain(drain, 0, VEDA_WAIT_LIMIT_NS);
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int wq = warp % 4, r0 = warp / 4 * R, key = tid & 127, half = key >> 6, kk = key & 63;
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16) + 4 * r0;  // this thread's lane and columns
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    bool ok = true;
    for (int e = 0; e < n_steps; ++e) {
      const int st = e % ST;
      // (this S was issued behind P V of step e-2, whose P is overwritten here)
      ok = mbar_wait(s_full + (e & 1), (e >> 1) & 1, abort_flag, g.dev_status);
      tc_fence_after();
      const StepMeta& sm = meta[st];
      uint32_t u[4 * R];
      tmem_load(lane_addr + (e & 1) * N, u);
      const float sk = sm.ks[half], ev = sm.ev[half];
      const int left = sm.left[half], pos = sm.pos[half] + kk;
      const bool full = sm.full, first = pos < p.sinks || p.window <= 0;
      float x[R];
      bool over = !ok;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float s = fmaf(fmaf(fmaf(__uint_as_float(u[3 * R + r]), 0.0625f, __uint_as_float(u[2 * R + r])), 0.0625f,
                                  __uint_as_float(u[R + r])), 0.0625f, __uint_as_float(u[r]));
        x[r] = fmaf(s, qs[r0 + r] * sk, ev);
        if (!full && !((pos <= seen_hi[r0 + r]) & ((pos > seen_lo[r0 + r]) | first) & (kk < left))) x[r] = -INFINITY;
        over |= x[r] > m[r] + MARGIN;
      }
      if (softmax_any<SM>(over)) {
        // given up by all threads or by none: the barriers below count them all
        if (softmax_any<SM>(!ok)) {
          ok = false;
          break;
        }
        // new references: the largest x so far, as integers that rank alike
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int i = __float_as_int(x[r] == x[r] ? x[r] : -INFINITY);
          const int v = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
          if (lane == r) red[wq * RP + r0 + r] = __int_as_float(v ^ ((v >> 31) & 0x7fffffff));
        }
        softmax_sync<SM>();
        float al[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float* v = red + r0 + r;
          const float mx = fmaxf(fmaxf(v[0], v[RP]), fmaxf(v[2 * RP], v[3 * RP]));
          const float mn = fmaxf(m[r], mx);
          al[r] = mn == m[r] ? 1.f : fast_exp2(m[r] - mn);
          m[r] = mn;
          l[r] *= al[r];
        }
        if (e > 0) {  // O, once P V of the last step has completed
          mbar_wait(free_ + (e - 1) % ST, ((e - 1) / ST) & 1, abort_flag, g.dev_status);
          __syncwarp();
          tc_fence_after();
          uint32_t o[4 * R];
          tmem_load(lane_addr + 2 * N, o);
#pragma unroll
          for (int k = 0; k < 4 * R; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al[k % R]);
          tmem_store(lane_addr + 2 * N, o);
        }
      }
      const float rv = sm.rv[half];
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const float p0 = fast_exp2(x[r] + (OFF - (m[r] == -INFINITY ? 0.f : m[r])));
        const float p1 = fast_exp2(x[r + 1] + (OFF - (m[r + 1] == -INFINITY ? 0.f : m[r + 1])));
        x[r] = p0;
        x[r + 1] = p1;
        // NaN scales reach the rows that see the tile through P, and no other
        l[r] += p0 == 0.f ? 0.f : p0 * rv;
        l[r + 1] += p1 == 0.f ? 0.f : p1 * rv;
        uint16_t c[4];
        four_parts(p0, p1, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = 4 * r0 + k * R + r;
          uint8_t* dst = smem + Cfg::OFF_P + (e & 1) * N * STEP + (key & 15);
          dst[n * 128 + (((key >> 4) ^ (n & 7)) << 4)] = (uint8_t)c[k];
          dst[(n + 1) * 128 + (((key >> 4) ^ ((n + 1) & 7)) << 4)] = (uint8_t)(c[k] >> 8);
        }
      }
      const int entry = sm.entry[half];
      if (!full) {
        // V rows behind the last token become zeroes: their codes may be anything
        if (sm.left[0] + sm.left[1] < STEP) {
          mbar_wait(v_full + st, (e / ST) & 1, abort_flag, g.dev_status);
          if (kk >= left && r0 == 0) {
            uint4* v = reinterpret_cast<uint4*>(smem + (st * 2 + 1) * Cfg::CB + key * D);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(p_full + (e & 1));
      if (p.lw && entry >= 0) {
        const int ppt = g.tile / 32;
        const long long piece = (long long)bh * p.pieces_cap + entry * ppt + (wq & (ppt - 1));
        float ref[R];
#pragma unroll
        for (int r = 0; r < R; ++r) ref[r] = m[r];
        warp_rows<R, 16>(x, ref, lane);
        const int r = r0 + lane / (32 / R);
        if (lane % (32 / R) == 0 && r < rows)
          p.lw[piece * p.rows_cap + r] = x[0] == 0.f ? -INFINITY : __log2f(x[0]) + (ref[0] - OFF - ev);
      }
    }
    if (n_steps > 0)  // the last P V (and with it all before), or after an abort whatever was issued
      ok = __all_sync(0xffffffffu,
                      mbar_wait(free_ + (n_steps - 1) % ST, ((n_steps - 1) / ST) & 1, abort_flag, g.dev_status) && ok);
    tc_fence_after();
    // row sums over the keys
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v = l[r];
#pragma unroll
      for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (lane == r) red[wq * RP + r0 + r] = v;
    }
    softmax_sync<SM>();
    uint32_t u[4 * R];
    if (n_steps > 0 && ok) {
      tmem_load(lane_addr + 2 * N, u);
    } else {
#pragma unroll
      for (int k = 0; k < 4 * R; ++k) u[k] = 0;
    }
    float o[R];  // this thread's channel of its rows
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float* v = red + r0 + r;
      l[r] = v[0] + v[RP] + v[2 * RP] + v[3 * RP];
      o[r] = fmaf(fmaf(fmaf(__uint_as_float(u[3 * R + r]), 0.0625f, __uint_as_float(u[2 * R + r])), 0.0625f,
                       __uint_as_float(u[R + r])), 0.0625f, __uint_as_float(u[r]));
    }
    // the rows' tokens, worked out before the wait for the other parts
    int tok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) tok[r] = (r0 + r) / p.group;
    bool last = true;
    if (parts > 1) {
      const long long row0 = ((long long)bh * p.splits + sp) * p.rows_pad + r0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r0 + r < rows && key < D) p.part_o[(row0 + r) * D + key] = o[r];
        if (r0 + r < rows && key == r) p.part_ml[row0 + r] = make_float2(m[r], l[r]);
      }
      softmax_sync<SM>();
      if (tid == 0) {  // releases the block's writes, acquires those of the blocks before
        int before;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrive + bh) : "memory");
        cnt[3] = before == parts - 1;
        if (before == parts - 1) p.arrive[bh] = 0;
      }
      softmax_sync<SM>();
      last = cnt[3] != 0;
      if (last) {
        // a warp per row: its parts' factors, then each thread its channel
        const float2* ml = p.part_ml + (long long)bh * p.splits * p.rows_pad;
        const float* po = p.part_o + ((long long)bh * p.splits * p.rows_pad + r0) * D + key;
        float* fac = reinterpret_cast<float*>(smem);  // [parts][RP], in the ring
        // parts whose O is in flight, the first of them beside the factors (as registers allow)
        constexpr int AHEAD = RP == 4 ? 8 : 16 / R;
        float v[AHEAD][R];
        auto fetch = [&](int s0) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
              v[u][r] = s0 + u < parts && r0 + r < rows && key < D
                            ? __ldcg(po + ((long long)(s0 + u) * p.rows_pad + r) * D)
                            : 0.f;
        };
        fetch(0);
        for (int r = warp; r < rows; r += SM / 32) {
          const float2 none = make_float2(-INFINITY, 0.f);
          const float2 x0 = lane < parts ? __ldcg(&ml[(long long)lane * p.rows_pad + r]) : none;
          float mx = x0.x, ls = 0.f;
          for (int s = lane + 32; s < parts; s += 32) mx = fmaxf(mx, __ldcg(&ml[(long long)s * p.rows_pad + r].x));
#pragma unroll
          for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          for (int s = lane; s < parts; s += 32) {
            const float2 x = s == lane ? x0 : __ldcg(&ml[(long long)s * p.rows_pad + r]);
            const float f = x.x == -INFINITY ? (x.y == x.y ? 0.f : 1.f) : fast_exp2(x.x - mx);
            fac[s * RP + r] = f;
            ls += x.y * f;
          }
#pragma unroll
          for (int d = 16; d; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
          if (lane == 0) {
            red[r] = mx;
            red[RP + r] = ls;
          }
        }
        softmax_sync<SM>();
#pragma unroll
        for (int r = 0; r < R; ++r) {
          m[r] = red[r0 + r];
          l[r] = red[RP + r0 + r];
          o[r] = 0.f;
        }
        for (int s0 = 0; s0 < parts; s0 += AHEAD) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u)
            if (s0 + u < parts)
#pragma unroll
              for (int r = 0; r < R; ++r) o[r] = fmaf(v[u][r], r0 + r < rows ? fac[(s0 + u) * RP + r0 + r] : 0.f, o[r]);
          if (s0 + AHEAD < parts) fetch(s0 + AHEAD);
        }
      }
    }
    if (last) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = r0 + r;
        if (row >= rows) break;
        const bool none = l[r] == 0.f;
        const int qh = h * p.group + row - tok[r] * p.group;
        if (key < D)
          p.o[b * p.o_sb + (long long)tok[r] * p.o_sn + (long long)qh * p.o_sh + key] =
              __float2bfloat16(none ? 0.f : o[r] / l[r]);
        if (key == r) {
          const float l2 = none ? -INFINITY : log2f(l[r]) + (m[r] == -INFINITY ? 0.f : m[r]) - OFF;
          if (p.lse) p.lse[((long long)b * p.heads + qh) * p.n_q + tok[r]] = l2 * LN2;
          qs[row] = l2;
        }
      }
      if (p.weight) {
        softmax_sync<SM>();
        // a thread per piece, those of a tile side by side
        const int ppt = g.tile / 32, pieces = nb * ppt;
        for (int base = 0; base < pieces; base += 2 * SM) {
          float v[2][RP], was[2];
          int ps[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int pc = base + u * SM + tid;
            const bool in = pc < pieces;
            ps[u] = in ? g.pos[trow + pc / ppt] : 0;
            was[u] = in && p.decay != 0.f ? p.weight[trow + pc / ppt] : 0.f;
            const float* lw = p.lw + ((long long)bh * p.pieces_cap + pc) * p.rows_cap;
#pragma unroll
            for (int r = 0; r < RP; ++r) v[u][r] = in && pc * 32 < total && r < rows ? __ldcg(lw + r) : -INFINITY;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int pc = base + u * SM + tid;
            float w = 0.f;
            if (kv_tile_seen(ps[u], g.tile, t_lo, t_hi, p.causal, p.window, p.sinks)) {
#pragma unroll
              for (int r = 0; r < RP; ++r) {
                const float z = r < rows ? qs[r] : 0.f;
                // none of it seen: nothing, even of a row that is NaN
                if (v[u][r] != -INFINITY && z != -INFINITY) w += fast_exp2(v[u][r] - z);
              }
            }
            for (int d = 1; d < ppt; d <<= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
            if (pc < pieces && pc % ppt == 0) p.weight[trow + pc / ppt] = p.decay == 0.f ? w : p.decay * was[u] + w;
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM);
  }
}

// Blocks sum the weights of one tile with many threads where tiles are few, and of
// four tiles where there are enough of them for every SM: the rows' sums are read
// once per block.
__host__ __device__ constexpr int finish_threads(int tiles) { return tiles == 1 ? 1024 : 256; }


// What is left behind the tile kernel, in one launch: a launch's latency is most of
// what either part takes (3 x 333 tokens, window 4,096: 39 us with a launch each,
// 36 with one).

// Parts of a row that are in flight together, and what has come of those before.
constexpr int PARTS_AHEAD = 4;
struct RowSum {
  float m = -INFINITY, l = 0.f;

  // Takes in the (reference, sum) pairs of parts; `mul` is what the parts before
  // have to be scaled by, f[u] what these have.
  __device__ __forceinline__ void add(const float2 (&x)[PARTS_AHEAD], float& mul, float (&f)[PARTS_AHEAD]) {
    float mx = m;
#pragma unroll
    for (int u = 0; u < PARTS_AHEAD; ++u) mx = fmaxf(mx, x[u].x);
    mul = mx == m ? 1.f : fast_exp2(m - mx);
    m = mx;
    l *= mul;
#pragma unroll
    for (int u = 0; u < PARTS_AHEAD; ++u) {
      // a part without a reference counts only where its sum is NaN
      f[u] = x[u].x == -INFINITY ? (x[u].y == x[u].y ? 0.f : 1.f) : fast_exp2(x[u].x - mx);
      l += x[u].y * f[u];
    }
  }
  __device__ __forceinline__ float lse2() const {
    return l == 0.f ? -INFINITY : log2f(l) + (m == -INFINITY ? 0.f : m) - OFF;
  }
};
__device__ __forceinline__ void load_parts(const float2* ml, long long stride, int s0, int parts,
                                           float2 (&x)[PARTS_AHEAD]) {
#pragma unroll
  for (int u = 0; u < PARTS_AHEAD; ++u)
    x[u] = s0 + u < parts ? ml[(s0 + u) * stride] : make_float2(-INFINITY, 0.f);
}

// Joins the parts of a row, D/4 lanes to a row.
template <int D>
__device__ __forceinline__ void join_row(const KvGeom& g, const KvAttnParams& p, int b, int h, int r, int c4) {
  const int bh = b * g.hkv + h;
  const long long stride = p.rows_pad;
  const float2* ml = p.part_ml + (long long)bh * p.parts * stride + r;
  const float* po = p.part_o + ((long long)bh * p.parts * stride + r) * D + c4 * 4;
  RowSum sum;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.parts; s0 += PARTS_AHEAD) {
    float2 x[PARTS_AHEAD];
    float4 v[PARTS_AHEAD];
    load_parts(ml, stride, s0, p.parts, x);
#pragma unroll
    for (int u = 0; u < PARTS_AHEAD; ++u)  // (a part without keys has written only its sum)
      v[u] = s0 + u < p.parts ? *reinterpret_cast<const float4*>(po + (s0 + u) * stride * D)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    float mul, f[PARTS_AHEAD];
    sum.add(x, mul, f);
    o.x *= mul;
    o.y *= mul;
    o.z *= mul;
    o.w *= mul;
#pragma unroll
    for (int u = 0; u < PARTS_AHEAD; ++u)
      if (f[u] != 0.f) {
        o.x += v[u].x * f[u];
        o.y += v[u].y * f[u];
        o.z += v[u].z * f[u];
        o.w += v[u].w * f[u];
      }
  }
  const float inv = sum.l == 0.f ? 0.f : 1.0f / sum.l;
  const int i = r / p.group, qh = h * p.group + r - i * p.group;
  *reinterpret_cast<uint2*>(p.o + b * p.o_sb + (long long)i * p.o_sn + (long long)qh * p.o_sh + c4 * 4) =
      make_uint2(pack_bf16x2_rn(o.x * inv, o.y * inv), pack_bf16x2_rn(o.z * inv, o.w * inv));
  if (c4 == 0 && p.lse) p.lse[((long long)b * p.heads + qh) * p.n_q + i] = sum.lse2() * LN2;
}

// The row's log2 normaliser from its parts, as join_row finds it.
__device__ __forceinline__ float row_lse2(const KvAttnParams& p, int bh, int r) {
  const float2* ml = p.part_ml + (long long)bh * p.parts * p.rows_pad + r;
  RowSum sum;
  for (int s0 = 0; s0 < p.parts; s0 += PARTS_AHEAD) {
    float2 x[PARTS_AHEAD];
    float mul, f[PARTS_AHEAD];
    load_parts(ml, p.rows_pad, s0, p.parts, x);
    sum.add(x, mul, f);
  }
  return sum.lse2();
}

// weight[tile] = decay * weight[tile] + sum over rows of 2^(lw - lse2), for TW
// tiles next to one another: a thread per row, the threads' sums joined in a
// fixed order.
template <int TW>
__device__ __forceinline__ void sum_weights(const KvGeom& g, const KvAttnParams& p, int b, int h, int i0, int nb,
                                            int rows, int t0, const int (&ps)[TW], float* part) {
  const int bh = b * g.hkv + h, tid = threadIdx.x, lane = tid % 32;
  constexpr int threads = finish_threads(TW);
  const float* lw = p.lw + ((long long)bh * p.pieces_cap + i0) * p.rows_cap;
  float w[TW];
#pragma unroll
  for (int k = 0; k < TW; ++k) w[k] = 0.f;
  constexpr int AHEAD = TW == 1 ? 4 : 2;  // rows whose loads are in flight
  for (int r0 = tid; r0 < rows; r0 += AHEAD * threads) {
    float x[AHEAD][TW], z[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int r = r0 + u * threads;
#pragma unroll
      for (int k = 0; k < TW; ++k) x[u][k] = r < rows && i0 + k < nb ? lw[(long long)k * p.rows_cap + r] : -INFINITY;
      z[u] = r >= rows ? -INFINITY : p.parts == 1 ? p.lse2[(long long)bh * p.rows_cap + r] : row_lse2(p, bh, r);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      // only tiles that a row tile's CTA could see were visited
      const int a = (r0 + u * threads) / p.tile_rows * p.tile_rows, c = min(rows, a + p.tile_rows) - 1;
      const int t_lo = t0 + a / p.group, t_hi = t0 + c / p.group;
#pragma unroll
      for (int k = 0; k < TW; ++k)
        // none of it seen: nothing, even of a row that is NaN
        if (z[u] != -INFINITY && x[u][k] != -INFINITY &&
            kv_tile_seen(ps[k], g.tile, t_lo, t_hi, p.causal, p.window, p.sinks))
          w[k] += fast_exp2(x[u][k] - z[u]);
    }
  }
#pragma unroll
  for (int k = 0; k < TW; ++k) {
#pragma unroll
    for (int d = 16; d; d >>= 1) w[k] += __shfl_xor_sync(0xffffffffu, w[k], d);
    if (lane == 0) part[tid / 32 * TW + k] = w[k];
  }
  __syncthreads();
  if (tid < TW && i0 + tid < nb) {
    float sum = 0.f;
#pragma unroll
    for (int y = 0; y < threads / 32; ++y) sum += part[y * TW + tid];
    float* dst = p.weight + (long long)bh * g.nb_cap + i0 + tid;
    *dst = p.decay == 0.f ? sum : p.decay * *dst + sum;
  }
}

template <int D, int TW>
__global__ void __launch_bounds__(finish_threads(TW), TW == 1 ? 1 : 5) kv_finish_kernel(const KvGeom g, const KvAttnParams p) {
  __shared__ float part[finish_threads(TW) / 32 * TW];
  const int h = blockIdx.y, b = blockIdx.z;
  const int i0 = (int)blockIdx.x < p.weight_blocks ? (int)blockIdx.x * TW : -1;  // negative: a block that joins
  int n_b, held, total, ps[TW];
  after_predecessor();
  const int t0 = g.next_pos[b];
#pragma unroll
  for (int k = 0; k < TW; ++k)
    ps[k] = i0 >= 0 && i0 + k < g.nb_cap ? g.pos[((long long)b * g.hkv + h) * g.nb_cap + i0 + k] : 0;
  const bool fine = kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total);
  const int rows = n_b * p.group;
  if (!fine || n_b == 0) return;
  if (i0 < 0) {
    constexpr int PER = finish_threads(TW) / (D / 4);  // rows at a time
    const int r0 = (blockIdx.x - p.weight_blocks) * p.join_rounds * PER + threadIdx.x / (D / 4);
    for (int y = 0; y < p.join_rounds && r0 + y * PER < rows; ++y)
      join_row<D>(g, p, b, h, r0 + y * PER, threadIdx.x % (D / 4));
  } else {
    const int nb = (total + g.tile - 1) / g.tile;
    bool seen = false;  // by any row
#pragma unroll
    for (int k = 0; k < TW; ++k)
      seen |= i0 + k < nb && kv_tile_seen(ps[k], g.tile, t0, t0 + n_b - 1, p.causal, p.window, p.sinks);
    if (i0 < nb) sum_weights<TW>(g, p, b, h, i0, nb, seen ? rows : 0, t0, ps, part);
  }
}

template <int D, int RP>
cudaError_t launch_rows_t(const KvGeom& g, const KvAttnParams& p, cudaStream_t s) {
  using Cfg = RowsCfg<D, RP>;
  KvMaps maps;
  const uint64_t rows = (uint64_t)g.n_slots * g.tile;
  if (encode_tensor_map_2d_u8(&maps.k, g.k8, D, rows, HALF) != CUDA_SUCCESS ||
      encode_tensor_map_2d_u8(&maps.v, g.v8, D, rows, HALF) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem((const void*)kv_attn_rows_kernel<D, RP>, Cfg::ALLOC, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kv_attn_rows_kernel<D, RP>, dim3(p.splits, g.hkv, g.B), Cfg::THREADS, Cfg::ALLOC, s, g, p, maps);
}

template <int D>
cudaError_t launch_rows(const KvGeom& g, const KvAttnParams& p, cudaStream_t s) {
  return p.rows_cap <= 4 ? launch_rows_t<D, 4>(g, p, s)
                         : p.rows_cap <= 8 ? launch_rows_t<D, 8>(g, p, s) : launch_rows_t<D, 16>(g, p, s);
}

}  // namespace

// Tokens that the rows of a row tile span.
static int n_tok(int rows, int group) { return (rows + group - 1) / group + 1; }

size_t kv_attn_plan(const KvGeom& g, KvAttnParams& p, bool weights, uint8_t* ws) {
  const long long rows = (long long)p.n_q * p.group;
  p.tiles = rows > FEW_ROWS;
  p.tile_rows = p.tiles ? 256 : FEW_ROWS;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  p.rows_cap = (int)rows;
  p.rows_pad = p.row_tiles * p.tile_rows;
  p.piece = p.tiles ? g.tile : 32;
  p.pieces_cap = g.nb_cap * (g.tile / p.piece);
  const long long ctas = (long long)g.B * g.hkv * p.row_tiles, keys = (long long)g.nb_cap * g.tile;
  p.splits = 1;
  p.alt = 0;
  if (p.tiles) {
    // One CTA per SM: waves of CTAs, each as long as its steps and what begins
    // and ends it; what is split is written and read once more and joined.
    // Measured at d = 128: 2.1 us a step, 5 us a CTA, 8 us for the join.
    // The workspace is asked for without a window, so one only lowers the split:
    // fewer steps alone could raise it, as the steps of a split are rounded up.
    p.alt = rows <= 128;
    const double t = (p.alt ? 1.1 : 2.1) * g.d / 128;
    auto split = [&](long long see, int most) {
      const double steps = (double)((see + 127) / 128);
      double best = 0;
      int at = 1;
      for (int s = 1; s <= most && (s == 1 || steps >= 3 * s); ++s) {
        const double waves = (double)((ctas * s + 147) / 148);
        const double us = waves * (ceil(steps / s) * t + 5) +
                          (s > 1 ? 8 + (double)ctas * s * (p.alt ? 2 * rows : p.tile_rows) * g.d * 8 / 4e6 : 0);
        if (s == 1 || us < best) {
          best = us;
          at = s;
        }
      }
      return at;
    };
    p.splits = split(keys, p.alt ? 16 : 32);
    const long long see = p.window > 0 ? (long long)p.window + p.sinks + n_tok(p.tile_rows, p.group) + 2 * g.tile : keys;
    if (see < keys) p.splits = split(see, p.splits);
  } else {
    // two CTAs per SM, each with a step at least
    const long long want = 296 / ctas, most = (keys + STEP - 1) / STEP;
    p.splits = (int)(want < most ? want : most);
    if (p.splits < 1) p.splits = 1;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = ws ? ws + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.parts = p.alt ? 2 * p.splits : p.splits;
  const size_t prows = (size_t)g.B * g.hkv * p.parts * p.rows_pad;
  p.part_ml = reinterpret_cast<float2*>(take(prows * 8));
  p.part_o = p.parts == 1 ? nullptr : reinterpret_cast<float*>(take(prows * g.d * 4));
  p.lse2 = nullptr;
  p.lw = nullptr;
  if (weights) {
    if (p.tiles) p.lse2 = reinterpret_cast<float*>(take((size_t)g.B * g.hkv * rows * 4));
    p.lw = reinterpret_cast<float*>(take((size_t)g.B * g.hkv * rows * p.pieces_cap * 4));
  }
  return off;
}

size_t kv_attn_ws_bytes(const KvGeom& g, int heads, int n_q, bool weights) {
  KvAttnParams p = {};
  p.heads = heads;
  p.group = heads / g.hkv;
  p.n_q = n_q;
  return kv_attn_plan(g, p, weights, nullptr);
}

cudaError_t launch_kv_attn(const KvGeom& g, KvAttnParams p, void* ws, cudaStream_t s) {
  kv_attn_plan(g, p, p.weight != nullptr, static_cast<uint8_t*>(ws));
  if (!p.tiles) return g.d == 128 ? launch_rows<128>(g, p, s) : launch_rows<64>(g, p, s);
  cudaError_t e = launch_kv_attn_tiles(g, p, s);
  if (e != cudaSuccess) return e;
  if (p.parts == 1 && !p.weight) return cudaSuccess;
  const bool four = (long long)g.nb_cap * g.hkv * g.B > 8 * 148;
  const int threads = finish_threads(four ? 4 : 1), per = threads / (g.d / 4);
  // weights first, as their blocks take longest; joins in up to 8 rounds of what the device holds
  const long long joins = p.parts == 1 ? 0 : (p.rows_cap + per - 1) / per, rounds = joins * g.hkv * g.B / (5 * 148);
  p.join_rounds = rounds < 1 ? 1 : rounds > 8 ? 8 : (int)rounds;
  p.weight_blocks = !p.weight ? 0 : four ? (g.nb_cap + 3) / 4 : g.nb_cap;
  const dim3 grid(p.weight_blocks + (unsigned)((joins + p.join_rounds - 1) / p.join_rounds), g.hkv, g.B);
  return launch_chained(g.d == 128 ? (four ? kv_finish_kernel<128, 4> : kv_finish_kernel<128, 1>)
                                   : (four ? kv_finish_kernel<64, 4> : kv_finish_kernel<64, 1>),
                        grid, threads, 0, s, g, p);
}

}  // namespace veda
