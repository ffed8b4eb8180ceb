// Attention over the 8-bit K/V tile cache, for many query rows (whole chunks
// and prompts): tcgen05 MMAs with accumulators in TMEM.
//
// A CTA owns two row tiles A and B of 128 query rows of one K/V head (row =
// token * group + head of the group) and walks the tiles that they see, 128
// keys a step.
//   S = Q K^T   kind::f8f6f4 on the codes as they lie in the cache: each Q row,
//               times a power of two, is the sum of two e4m3 parts (8 bits, as
//               bf16 has; values below 2^-10 of the row's largest lose what is
//               below 2^-18 of it), so K needs no conversion and two passes at
//               the 8-bit rate cost what one at 16 bits does.
//   O += P V    kind::f16: P as fp16 in TMEM (see kv_attn.cu for the exponent
//               that carries the V scale), V converted from e4m3 by two
//               warps of their own; a second e4m3 part of P would cost the softmax
//               warps, which bound the kernel, more than this costs those.
// Where a head has no more rows than one tile (p.alt), B has the same rows as A
// and takes every second step: two chains of softmax and MMAs per SM instead of
// one, each a part of its own for the join.
// The softmax reference is the first maximum and moves only where a step's sum
// passes 2^15 (then P may no longer fit fp16).
//
// Roles (384 threads; more would leave the softmax too few registers for a row of S):
//   warps 0-3 / 4-7  softmax of A / B: a thread owns a row (TMEM lane). S_A in
//                    TMEM columns [0,128), S_B [128,256); P over the second
//                    half of its S; O_A at [256,256+D), O_B at [384,384+D).
//   warp 8           producer: table, scales, TMA copies of the K and V codes
//   warp 9           MMA issuer (one thread)
//   warps 10, 11     V: e4m3 tile -> fp16 tile
// Every wait is bounded, as in the other pipelines.
// Measured: 3,840 x 34,560, 24 heads, d = 128: 1.68 ms, 970 TFLOP/s (a step of 256
// rows x 128 keys takes ~3,680 clocks against 2,048 of MMA; the clock is held at
// ~1.7 GHz by power); 2,048-token causal prompt, 32/8 heads: 65 us.
#include "kv_attn.cuh"

namespace veda {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int KST = 3, VST = 2, WST = 2;  // stages: K codes, V codes, V fp16
// A description's slot is written again only after step_done of four steps
// later, whose S was issued behind the P of this step and of the row tile's next.
constexpr int MST = KST + 4;
constexpr int SDR = 4;                 // step-done barriers
constexpr float OVERFLOW_SUM = 32768.f;
constexpr int THREADS = 384, CONVERT_WARPS = 2;
// 2*128*208 + 128*88 = 64,512 = the 384*168 of the launch
constexpr int REGS_SOFTMAX = 208, REGS_ROLES = 88;

template <int D>
struct TileLayout {
  static constexpr int QB = BM * D;      // bytes of one part of a row tile
  static constexpr int CB = BN * D;      // bytes of a step's K or V codes
  static constexpr int WB = BN * D * 2;  // bytes of a step's V in fp16
  static constexpr int OFF_Q = 0;        // A hi, A lo, B hi, B lo
  static constexpr int OFF_K = 4 * QB;
  static constexpr int OFF_V = OFF_K + KST * CB;
  static constexpr int OFF_W = OFF_V + VST * CB;
  static constexpr int OFF_META = OFF_W + WST * WB;
  static constexpr int OFF_BAR = OFF_META + MST * (int)sizeof(StepMeta);
  static constexpr int NUM_BARS = KST + 2 * VST + WST + SDR + 2 + 2 + 2 + 1;  // and one per softmax warp
  static constexpr int OFF_MISC = OFF_BAR + (NUM_BARS + 8) * 8;
  static constexpr int ALLOC = OFF_MISC + 32 + 1024;
};
static_assert(sizeof(StepMeta) % 8 == 0, "barriers follow");

// `bytes` (a multiple of 16) of a row to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, int bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Token and head-of-group of a row, kept along as rows advance by a few (without a
// loop, so that the accesses of several rows overlap).
struct RowStep {
  int tok, gh, d_tok, d_gh, group;
  __device__ __forceinline__ RowStep(int row, int by, int group_) : group(group_) {
    tok = row / group;
    gh = row - tok * group;
    d_tok = by / group;
    d_gh = by - d_tok * group;
  }
  __device__ __forceinline__ void advance() {
    gh += d_gh;
    tok += d_tok;
    const bool over = gh >= group;
    gh -= over ? group : 0;
    tok += over;
  }
};

// The keys of one half that the query at position t sees, as bits.
__device__ __forceinline__ uint64_t half_seen(const KvAttnParams& p, int t, int pos, int left) {
  auto below = [](long long n) { return n >= HALF ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull; };
  const long long d = (long long)t - pos;
  uint64_t seen = below(left);
  if (p.causal) seen &= below(d + 1);
  if (p.window > 0) seen &= ~below(d - p.window + 1) | below((long long)p.sinks - pos);
  return seen;
}

__device__ __forceinline__ void half_mask(uint32_t (&u)[64], uint64_t seen) {
  const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    if (!(lo >> k & 1u)) u[k] = 0xff800000u;
    if (!(hi >> k & 1u)) u[32 + k] = 0xff800000u;
  }
}

__device__ __forceinline__ float half_max(const uint32_t (&u)[64]) {
  float pm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) pm[i] = fmaxf(__uint_as_float(u[i]), __uint_as_float(u[8 + i]));
#pragma unroll
  for (int c = 16; c < 64; c += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) pm[i] = fmax3(pm[i], __uint_as_float(u[c + i]), __uint_as_float(u[c + 8 + i]));
  return fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
}

// P = 2^(s*c + nm) of one half as fp16 pairs; returns the sum of the fp32 values.
__device__ __forceinline__ float half_p(const uint32_t (&u)[64], float c, float nm, uint32_t (&pk)[32]) {
  const uint64_t C2 = f2(c, c), NM = f2(nm, nm);
  uint64_t acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = f2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const uint64_t x = f2_fma(f2(__uint_as_float(u[2 * w]), __uint_as_float(u[2 * w + 1])), C2, NM);
    float x0, x1;
    f2_split(x, x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    acc[w & 3] = f2_add(acc[w & 3], f2(p0, p1));
    pk[w] = pack_f16x2(p0, p1);
  }
  float lo, hi;
  f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
  return lo + hi;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    kv_attn_tiles_kernel(const KvGeom g, const KvAttnParams p, const __grid_constant__ KvMaps maps) {
  using Lay = TileLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int q_abort[8];
  __shared__ int sm_cnt[4];  // of kv_range, and the steps
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // Under a causal mask the last row tiles have the most keys, so every head's
  // start first (2,048-token prompt, 8 heads: 93 -> 77 us). Without one they are
  // equal, and a head's row tiles run together, so that its K and V come from
  // L2 (3,840 x 34,560, 24 heads: 1.70 against 1.64 ms the other way round).
  const int sp = blockIdx.x % p.splits, rest = blockIdx.x / p.splits, b = blockIdx.z;
  const int h = p.causal ? rest % g.hkv : rest / p.row_tiles;
  const int mt = p.row_tiles - 1 - (p.causal ? rest / g.hkv : rest % p.row_tiles);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int n_b, held, total;
  const int t0 = g.next_pos[b];
  const bool fits = kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total);
  const int rows = fits ? n_b * p.group : 0;
  const int base = mt * 2 * BM;
  if (p.fill && sp == 0) fill_rows<D>(p, b, h, max(base, rows), min(base + 2 * BM, p.rows_cap), tid, THREADS);
  if (base >= rows) return;
  const bool alt = p.alt, has_b = base + BM < rows || alt;
  const int bh = b * g.hkv + h;
  const long long trow = (long long)bh * g.nb_cap;
  const int t_lo = t0 + base / p.group, t_hi = t0 + (min(rows, base + 2 * BM) - 1) / p.group;

  // Q, a row per D/8 lanes: a warp reads and later writes whole rows. Lane
  // group `sub` has rows sub, sub + RPI, ... of the warp's 32.
  constexpr int LPR = D / 8, RPI = 32 / LPR, ITERS = 32 / RPI;
  const int rt = warp / 4, wrow = base + (alt ? warp % 4 : warp) * 32, sub = lane / LPR, c8 = lane % LPR;
  uint8_t* own = smem + Lay::OFF_Q + rt * 2 * Lay::QB;  // the row tile's Q, and its O at the end
  const bool mine = warp < 4 || (warp < 8 && has_b);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* k_full = bars;
  uint64_t* v_full = k_full + KST;
  uint64_t* v_free = v_full + VST;   // an arrival per converting warp: it has read the codes
  uint64_t* w_full = v_free + VST;   // an arrival per converting warp
  uint64_t* step_done = w_full + WST;  // S of step e and P V of e-1 have completed
  uint64_t* s_full = step_done + SDR;     // [2]
  uint64_t* p_full = s_full + 2;          // [2], 128 arrivals
  uint64_t* pv_done = p_full + 2;         // [2]
  uint64_t* drain = pv_done + 2;
  uint64_t* q_full = drain + 1;  // [8], the softmax warps' own
  StepMeta* meta = reinterpret_cast<StepMeta*>(smem + Lay::OFF_META);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::OFF_MISC + 4);
  // A softmax warp's rows of Q, a copy each, to where V in fp16 will be: under way
  // while the steps are found (2,048-token prompt: loads to registers, a batch of
  // rows ahead, 66.0 us, copies 64.8).
  uint8_t* q_raw = smem + Lay::OFF_W + warp * 32 * 2 * D;
  bool ok = true;  // (the softmax warps')
  if (mine) {
    if (lane == 0) {
      q_abort[warp] = 0;
      mbar_init(q_full + warp, 1);
      fence_mbar_init();
      mbar_expect_tx(q_full + warp, max(0, min(32, rows - wrow)) * 2 * D);
    }
    __syncwarp();
    if (wrow + lane < rows) {
      const int tok = (wrow + lane) / p.group, gh = wrow + lane - tok * p.group;
      bulk_load(q_raw + lane * 2 * D, p.q.p + b * p.q.sb + (long long)tok * p.q.sn + (long long)(h * p.group + gh) * p.q.sh,
                2 * D, q_full + warp);
    } else {
#pragma unroll 1
      for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(q_raw + lane * 2 * D + c * 16) = make_uint4(0, 0, 0, 0);
    }
  }

  // The steps are worked out by the warps that do not take Q apart meanwhile.
  KvRange rg{0, 0, 0};
  int s_lo = 0, n_steps = 0;
  if (warp >= 8) {
    auto sync = [] { asm volatile("bar.sync 2, 128;" ::: "memory"); };
    if (p.window > 0 || p.causal) {
      if (tid < 256 + 3) sm_cnt[tid - 256] = 0;
      sync();
    }
    const int nb = (total + g.tile - 1) / g.tile;
    rg = kv_range(g, p, trow, nb, t_lo, t_hi, t0 + n_b - 1, sm_cnt, tid - 256, 128, sync);
    const int steps_all = (rg.count() * g.tile + BN - 1) / BN;
    const int per = (steps_all + p.splits - 1) / p.splits;
    s_lo = min(steps_all, sp * per);
    n_steps = min(steps_all, s_lo + per) - s_lo;
    if (tid == 256) sm_cnt[3] = n_steps;
  }

  // Each role prepares its part before the one barrier: the first copies are
  // under way while Q is taken apart.
  StepFeed feed;
  int fed = 0;             // steps whose K copies were issued (the producer's)
  int v_row0 = 0, v_row1 = 0;  // pool rows of the step whose V comes next
  auto load_half = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int row0, int row1) {
    if (lane == 0) {
      mbar_expect_tx(bar, (row0 >= 0 ? Lay::CB / 2 : 0) + (row1 >= 0 ? Lay::CB / 2 : 0));
      if (row0 >= 0) tma_load_2d(dst, map, bar, 0, row0);
      if (row1 >= 0) tma_load_2d(dst + Lay::CB / 2, map, bar, 0, row1);
    }
    __syncwarp();
  };
  auto produce_k = [&](int e, int& row0, int& row1) {
    if ((e & 15) == 0) feed.load(g, trow, rg, total, s_lo, e, n_steps, lane);
    feed.put(meta[e % MST], g, p, e, t_lo, t_hi, lane, row0, row1);
    __syncwarp();
    load_half(&maps.k, k_full + e % KST, smem + Lay::OFF_K + e % KST * Lay::CB, row0, row1);
  };
  auto produce_v = [&](int e, int row0, int row1) {
    load_half(&maps.v, v_full + e % VST, smem + Lay::OFF_V + e % VST * Lay::CB, row0, row1);
  };
  float qs = 0.f;
  if (warp == 8) {
    if (lane < Lay::NUM_BARS) {
      uint64_t* bar = bars + lane;
      mbar_init(bar, bar >= v_free && bar < w_full + WST ? CONVERT_WARPS : bar == p_full || bar == p_full + 1 ? 128 : 1);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    __syncwarp();
    // K runs a step ahead of V: V waits for the conversion of an earlier one
    if (n_steps > 0) produce_k(0, v_row0, v_row1);
    fed = 1;
  } else if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  } else if (mine) {
    // Q in its two e4m3 parts, a few rows at a time: their chains of shuffles and
    // conversions overlap.
    constexpr int BATCH = 4;
    __syncwarp();
    ok = __all_sync(0xffffffffu, mbar_wait(q_full + warp, 0, q_abort + warp, g.dev_status));
    if (!ok) mbar_wait_drain(q_full + warp, 0, VEDA_WAIT_LIMIT_NS);
#pragma unroll 1
    for (int j0 = 0; j0 < ITERS; j0 += BATCH) {
      uint4 qw[BATCH];
      uint32_t top[BATCH];
#pragma unroll
      for (int y = 0; y < BATCH; ++y) {
        qw[y] = *reinterpret_cast<const uint4*>(q_raw + ((j0 + y) * RPI + sub) * 2 * D + c8 * 16);
        top[y] = max(max(bf16x2_top(qw[y].x), bf16x2_top(qw[y].y)), max(bf16x2_top(qw[y].z), bf16x2_top(qw[y].w)));
      }
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1)
#pragma unroll
        for (int y = 0; y < BATCH; ++y) top[y] = max(top[y], __shfl_xor_sync(0xffffffffu, top[y], d));
      uint32_t hi[BATCH][2], lo[BATCH][2];
#pragma unroll
      for (int y = 0; y < BATCH; ++y) {
        float mul, inv;
        q_scale<7>(top[y], mul, inv);
        mul = copysignf(mul, p.scale_log2);
        split_e4m3x4(qw[y].x, qw[y].y, mul, hi[y][0], lo[y][0]);
        split_e4m3x4(qw[y].z, qw[y].w, mul, hi[y][1], lo[y][1]);
        // the lane that owns the row keeps its factor
        const float got = __shfl_sync(0xffffffffu, inv, (lane % RPI) * LPR);
        if (lane / RPI == j0 + y) qs = got;
      }
#pragma unroll
      for (int y = 0; y < BATCH; ++y) {
        const int to = code_at<D>((warp % 4) * 32 + (j0 + y) * RPI + sub, c8 >> 1) + (c8 & 1) * 8;
        *reinterpret_cast<uint2*>(own + to) = make_uint2(hi[y][0], hi[y][1]);
        *reinterpret_cast<uint2*>(own + Lay::QB + to) = make_uint2(lo[y][0], lo[y][1]);
      }
    }
    qs *= fabsf(p.scale_log2);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  n_steps = sm_cnt[3];

  if (warp >= 8) {
    regs_lower<REGS_ROLES>();
    if (warp == 8) {
      // --------------------------------------------------------- producer
      int e = 0;  // V copies issued; K is at fed
      for (; e < n_steps; ++e) {
        int row0 = -1, row1 = -1;
        bool ok = true;
        if (fed < n_steps) {
          // the description's slot is free too, see MST
          ok = fed < KST || mbar_wait(step_done + (fed - KST) % SDR, ((fed - KST) / SDR) & 1, abort_flag, g.dev_status);
          if (!__all_sync(0xffffffffu, ok)) break;
          produce_k(fed++, row0, row1);
        }
        ok = e < VST || mbar_wait(v_free + e % VST, (e / VST - 1) & 1, abort_flag, g.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        produce_v(e, v_row0, v_row1);
        v_row0 = row0;
        v_row1 = row1;
      }
      if (*abort_flag && lane == 0) {  // let every copy that was started land
        for (int x = max(0, fed - KST); x < min(fed, n_steps); ++x)
          mbar_wait_drain(k_full + x % KST, (x / KST) & 1, VEDA_WAIT_LIMIT_NS);
        for (int x = max(0, e - VST); x < e; ++x)
          mbar_wait_drain(v_full + x % VST, (x / VST) & 1, VEDA_WAIT_LIMIT_NS);
      }
    } else if (warp == 9) {
      if (lane == 0) {
      // ------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_fmt0(BM, BN, false, false);
      constexpr uint32_t idesc_o = idesc_fmt0(BM, D, false, true);
      const uint64_t dQ = sdesc_codes<D>(smem_u32(smem + Lay::OFF_Q));
      const uint64_t dK = sdesc_codes<D>(smem_u32(smem + Lay::OFF_K));
      const uint64_t dW = sdesc_sw128(smem_u32(smem + Lay::OFF_W), BN * 128, 1024);
      bool ok = true;
      const int tiles = has_b ? 2 : 1;
      const int back = alt ? 2 : 1;  // a row tile's steps are so far apart
      auto issue_pv = [&](int r, int e) -> bool {  // P V of step e
        const int ws = e % WST;
        if (!mbar_wait(p_full + r, (alt ? e >> 1 : e) & 1, abort_flag, g.dev_status)) return false;
        if (!mbar_wait(w_full + ws, (e / WST) & 1, abort_flag, g.dev_status)) return false;
        tc_fence_after();
        const uint32_t o_addr = tmem + 2 * BN + r * BN, p_addr = tmem + r * BN + 64;
        const uint64_t d = dW + (uint64_t)(ws * (Lay::WB >> 4));
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_bf16_ts(o_addr, p_addr + kk * 8, d + (uint64_t)(kk * (2048 >> 4)), idesc_o, (e >= back || kk > 0) ? 1u : 0u);
        if (e + back >= n_steps) umma_commit(pv_done + r);
        return true;
      };
      for (int e = 0; ok && e < n_steps; ++e) {
        const int st = e % KST;
        if (!mbar_wait(k_full + st, (e / KST) & 1, abort_flag, g.dev_status)) break;
        tc_fence_after();
        for (int r = 0; r < tiles; ++r) {
          if (alt && r != (e & 1)) continue;
          if (e >= back && !(ok = issue_pv(r, e - back))) break;
          const uint64_t q = dQ + (uint64_t)(r * (2 * Lay::QB >> 4)), k = dK + (uint64_t)(st * (Lay::CB >> 4));
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8_ss(tmem + r * BN, q + (uint64_t)((part * Lay::QB + kk * 32) >> 4), k + (uint64_t)(kk * 32 >> 4),
                         idesc_s, (part || kk) ? 1u : 0u);
          umma_commit(s_full + r);
        }
        if (!ok) break;
        umma_commit(step_done + e % SDR);
      }
      // what is left: each row tile's last step
      for (int r = 0; r < tiles && ok && !*abort_flag; ++r) {
        const int e = alt ? n_steps - 1 - ((n_steps - 1 - r) & 1) : n_steps - 1;
        if (e >= 0) ok = issue_pv(r, e);
      }
      umma_commit(drain);
      mbar_wait_drain(drain, 0, VEDA_WAIT_LIMIT_NS);
      }
    } else {
    // ---------------------------------------------------------- V to fp16
    // a thread's 16 codes of one key become two 16-byte chunks of that key's
    // row in a 64-column box; eight threads next to one another take four
    // chunks of two keys, whose writes fall into different banks
    const int ct = tid - 320;
    constexpr int CH = D / 16, CT = CONVERT_WARPS * 32, VECS = BN * CH / CT;
    for (int e = 0; e < n_steps; ++e) {
      const int vt = e % VST, ws = e % WST;
      bool ok = mbar_wait(v_full + vt, (e / VST) & 1, abort_flag, g.dev_status);
      // fp16 slot: P V of step e - WST has completed
      if (ok && e >= WST) {
        const int sd = e - WST + (alt ? 2 : 1);
        ok = mbar_wait(step_done + sd % SDR, (sd / SDR) & 1, abort_flag, g.dev_status);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      const int left0 = meta[e % MST].left[0], left1 = meta[e % MST].left[1];
      const uint8_t* src = smem + Lay::OFF_V + vt * Lay::CB;
      uint8_t* dst = smem + Lay::OFF_W + ws * Lay::WB;
      constexpr int BATCH = 8;  // loads in flight
#pragma unroll
      for (int j0 = 0; j0 < VECS; j0 += BATCH) {
        uint4 c[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int x = (j0 + j) * CT + ct, quad = x >> 3;
          const int r = (quad / (CH / 4)) * 2 + ((x >> 2) & 1), ch = (quad % (CH / 4)) * 4 + (x & 3);
          c[j] = *reinterpret_cast<const uint4*>(src + code_at<D>(r, ch));
          // codes behind the last token may be anything
          if ((r & (HALF - 1)) >= (r < HALF ? left0 : left1)) c[j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int x = (j0 + j) * CT + ct, quad = x >> 3;
          const int r = (quad / (CH / 4)) * 2 + ((x >> 2) & 1), ch = (quad % (CH / 4)) * 4 + (x & 3);
          uint4 lo, hi;
          codes_f16(c[j].x, lo.x, lo.y);
          codes_f16(c[j].y, lo.z, lo.w);
          codes_f16(c[j].z, hi.x, hi.y);
          codes_f16(c[j].w, hi.z, hi.w);
          uint8_t* box = dst + (ch >> 2) * (BN * 128) + r * 128;
          const int c2 = (ch & 3) * 2;
          *reinterpret_cast<uint4*>(box + ((c2 ^ (r & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(box + (((c2 + 1) ^ (r & 7)) << 4)) = hi;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(v_free + vt);
        mbar_arrive(w_full + ws);
      }
    }
    }
  } else {
    regs_raise<REGS_SOFTMAX>();
    // ------------------------------------------------------------ softmax
    const int row = wrow + lane;
    const bool row_valid = row < rows;
    const int tok = row / p.group, t = t0 + tok;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const uint32_t s_col = rt * BN, o_col = 2 * BN + rt * BN;
    float m = -INFINITY, l = 0.f;
    if (!ok) *abort_flag = 1;
    const int first = alt ? rt : 0, stride = alt ? 2 : 1;
    const int n_mine = mine ? (n_steps - first + stride - 1) / stride : 0;  // steps of this row tile
    for (int j = 0; ok && j < n_mine; ++j) {
      const int e = first + j * stride;
      if (!__all_sync(0xffffffffu, mbar_wait(s_full + rt, j & 1, abort_flag, g.dev_status))) { ok = false; break; }
      if (wrow >= rows) {  // none of the warp's rows is one: its P may be anything
        mbar_arrive(p_full + rt);
        continue;
      }
      tc_fence_after();
      const StepMeta& sm = meta[e % MST];
      float c0 = qs * sm.ks[0], c1 = qs * sm.ks[1], ev0 = sm.ev[0], ev1 = sm.ev[1];
      const bool full = sm.full;
      uint64_t seen0 = 0, seen1 = 0;
      if (!full) {
        // a hidden key's logit is -inf, which the coefficient must leave so: it
        // is not 0, and a NaN one only counts where the row sees the half
        seen0 = half_seen(p, t, sm.pos[0], sm.left[0]);
        seen1 = half_seen(p, t, sm.pos[1], sm.left[1]);
        if (!seen0 || c0 == 0.f) c0 = 1e-37f;
        if (!seen1 || c1 == 0.f) c1 = 1e-37f;
        if (!seen0) ev0 = 0.f;
        if (!seen1) ev1 = 0.f;
      }
      uint32_t u[BN], pk0[32], pk1[32];
      uint32_t (&u0)[64] = *reinterpret_cast<uint32_t(*)[64]>(&u[0]);
      uint32_t (&u1)[64] = *reinterpret_cast<uint32_t(*)[64]>(&u[64]);
      float sum0, sum1;
      float alpha = 1.f;
      bool move = m == -INFINITY;  // the reference has to be found; in a second pass: found again
      for (int pass = 0;; ++pass) {
        tmem_ld128(lane_addr + s_col, u);  // P is not stored yet, so S is intact in a second pass
        if (!full) {
          half_mask(u0, seen0);
          half_mask(u1, seen1);
        }
        if (__any_sync(0xffffffffu, move)) {
          const float mx = fmaxf(half_max(u0) * c0 + ev0, half_max(u1) * c1 + ev1);
          const float m_new = move ? fmaxf(m, mx) : m;
          alpha = m_new == m ? 1.f : fast_exp2(m - m_new);
          m = m_new;
        }
        const float bias = OFF - (m == -INFINITY ? 0.f : m);
        sum0 = half_p(u0, c0, ev0 + bias, pk0);
        sum1 = half_p(u1, c1, ev1 + bias, pk1);
        move = !(sum0 + sum1 <= OVERFLOW_SUM);
        if (pass == 1 || !__any_sync(0xffffffffu, move)) break;
      }
      if (__any_sync(0xffffffffu, alpha != 1.f && l != 0.f)) {
        // O holds P V of all earlier steps: S of this one was issued behind them
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(lane_addr + o_col + c * 32, o);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
          tmem_st32(lane_addr + o_col + c * 32, o);
        }
      }
      l *= alpha;
      tmem_st32_async(lane_addr + s_col + 64, pk0);
      tmem_st32_async(lane_addr + s_col + 96, pk1);
      tmem_wait_st_keep(pk0, pk1);
      tc_fence_before();
      mbar_arrive(p_full + rt);
      l += (sum0 == 0.f ? 0.f : sum0 * sm.rv[0]) + (sum1 == 0.f ? 0.f : sum1 * sm.rv[1]);
      if (p.lw && row_valid) {
        // a tile of 128 is the whole step, of 64 half of it
        const float off = (m == -INFINITY ? 0.f : m) - OFF;
        float* dst = p.lw + (long long)bh * p.pieces_cap * p.rows_cap + row;
        auto put = [&](int x, float sum) {
          if (sm.entry[x] >= 0)
            dst[(long long)sm.entry[x] * p.rows_cap] = sum == 0.f ? -INFINITY : __log2f(sum) + (off - sm.ev[x]);
        };
        if (g.tile == BN) {
          put(0, sum0 + sum1);
        } else {
          put(0, sum0);
          put(1, sum1);
        }
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // O / l, or this split's part of them
    const long long part = (long long)bh * p.parts + (alt ? 2 * sp + rt : sp), prow = part * p.rows_pad + row;
    bool have = false;
    if (ok && n_mine > 0) {
      have = __all_sync(0xffffffffu, mbar_wait(pv_done + rt, 0, abort_flag, g.dev_status));
      tc_fence_after();
    }
    if (mine) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int qh = h * p.group + row - tok * p.group;
      // rows go through the row tile's own shared memory, 2 D bytes of each at
      // a time, so that a warp writes whole rows: its bf16 row, or half of its
      // fp32 one
      constexpr int UNITS = D / 8;  // 16-byte units per row and pass
      uint8_t* mem = own + (warp % 4) * 32 * 2 * D;
      auto slot = [&](int r, int u) { return mem + r * 2 * D + ((u ^ (r & (UNITS - 1))) << 4); };
      // a part without keys is no more than its sum, which is 0
      const int passes = p.parts == 1 ? 1 : n_steps ? 2 : 0;
      for (int ps = 0; ps < passes; ++ps) {
        const int cols = D >> (passes - 1);
        for (int c = 0; c < cols; c += 32) {
          uint32_t u[32];
          if (have) {
            tmem_ld32(lane_addr + o_col + ps * cols + c, u);
          } else {
#pragma unroll
            for (int y = 0; y < 32; ++y) u[y] = 0u;
          }
          if (passes == 2) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              *reinterpret_cast<uint4*>(slot(lane, c / 4 + y)) =
                  make_uint4(u[4 * y], u[4 * y + 1], u[4 * y + 2], u[4 * y + 3]);
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t x[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                x[z] = pack_bf16x2_rn(l == 0.f ? 0.f : __uint_as_float(u[8 * y + 2 * z]) * inv,
                                      l == 0.f ? 0.f : __uint_as_float(u[8 * y + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(slot(lane, c / 8 + y)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        }
        __syncwarp();
        static_assert(UNITS == LPR, "rows are written as Q was read");
        RowStep at(wrow + sub, RPI, p.group);
#pragma unroll 4
        for (int j = 0; j < ITERS; ++j) {
          const int r = j * RPI + sub;
          const uint4 v = *reinterpret_cast<const uint4*>(slot(r, c8));
          if (wrow + r < rows) {
            if (passes == 2) {
              const long long pr = part * p.rows_pad + wrow + r;
              *reinterpret_cast<uint4*>(p.part_o + pr * D + ps * (D / 2) + c8 * 4) = v;
            } else {
              *reinterpret_cast<uint4*>(p.o + b * p.o_sb + (long long)at.tok * p.o_sn +
                                        (long long)(h * p.group + at.gh) * p.o_sh + c8 * 8) = v;
            }
          }
          at.advance();
        }
        __syncwarp();
      }
      if (row_valid) {
        if (p.parts > 1) {
          p.part_ml[prow] = make_float2(m, l);
        } else {
          const float l2 = l == 0.f ? -INFINITY : log2f(l) + (m == -INFINITY ? 0.f : m) - OFF;
          if (p.lse) p.lse[((long long)b * p.heads + qh) * p.n_q + tok] = l2 * LN2;
          if (p.lse2) p.lse2[(long long)bh * p.rows_cap + row] = l2;
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const KvGeom& g, const KvAttnParams& p, cudaStream_t s) {
  KvMaps maps;
  const uint64_t rows = (uint64_t)g.n_slots * g.tile;
  if (encode_tensor_map_2d_u8(&maps.k, g.k8, D, rows, HALF) != CUDA_SUCCESS ||
      encode_tensor_map_2d_u8(&maps.v, g.v8, D, rows, HALF) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem((const void*)kv_attn_tiles_kernel<D>, TileLayout<D>::ALLOC, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kv_attn_tiles_kernel<D>, dim3(g.hkv * p.splits * p.row_tiles, 1, g.B), THREADS,
                        TileLayout<D>::ALLOC, s, g, p, maps);
}

}  // namespace

cudaError_t launch_kv_attn_tiles(const KvGeom& g, const KvAttnParams& p, cudaStream_t s) {
  return g.d == 128 ? launch<128>(g, p, s) : launch<64>(g, p, s);
}

}  // namespace veda
