// Attention over the 8-bit K/V tile cache, for few query rows.
//
// Row r of a K/V head is query token r / group, query head h*group + r % group.
// With c the codes, s the tile scales and x_ij = scale*log2(e) * (q_i . ck_j)
// * sk + log2(sv):
//   P_ij = 2^(x_ij - M_i + OFF),  O_i = sum_j P_ij cv_j / sum_j P_ij / sv.
// The V scale is part of the exponent, so P V runs on the bare codes and tiles
// of any scale add up in one accumulator; dividing P by sv again for the sum is
// exact for powers of two. M is a reference, not the maximum: it moves only
// when some x passes it by MARGIN, so that P stays within 2^(MARGIN + OFF) and
// fp16 (which has 11 bits of significand against bf16's 8, and is what an e4m3
// pair converts to in one instruction) holds it. OFF keeps what lies 2^-31
// below the reference out of fp16's zero: even a million such keys add less
// than a part in a thousand. Sums, references and O are fp32.
#include <cmath>

#include "kv_attn.cuh"

namespace veda {
namespace {

constexpr int ROWS = 16;    // query rows per CTA (the M of one mma)
constexpr int PIECE = 32;   // keys a warp takes at a time
constexpr int WARPS = 4;
constexpr int TILE_KERNEL_ROWS = 32;  // more query rows per K/V head than this: the tile kernel
constexpr float MARGIN = 8.f;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A CTA has 16 query rows of one K/V head and a range of its tiles, in pieces
// of 32 keys; warp w takes every fourth piece and keeps its own reference, sum
// and O, so that no warp waits for another before the end. Pieces reach the
// warp through its own ring of STAGES TMA copies on mbarriers: the bound is HBM
// (1 byte per K and V value, each used by up to 16 rows), so what matters is
// that enough copies are in flight, not which warp asks for them. Table
// entries, positions and scales of the warp's next 32 pieces sit in its lanes.
template <int D>
struct RowsCfg {
  static constexpr int STAGES = D == 128 ? 2 : 3;
  static constexpr int PB = PIECE * D;                                   // bytes of a piece of K or V
  static constexpr int SMEM = WARPS * STAGES * 2 * PB + 1024;            // and alignment
  static constexpr int CTAS = D == 128 ? 3 : 4;                          // per SM, by registers
};

template <int D>
__global__ void __launch_bounds__(WARPS * 32, RowsCfg<D>::CTAS)
    kv_attn_rows_kernel(const KvGeom g, const KvAttnParams p, const __grid_constant__ KvMaps maps) {
  using Cfg = RowsCfg<D>;
  constexpr int KS = D / 16;  // 16-wide steps over the head dimension
  constexpr int ST = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
  __shared__ int sm_cnt[3];
  __shared__ int sm_abort;
  __shared__ __align__(8) uint64_t bars[WARPS][ST];
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  const int mt = blockIdx.x % p.row_tiles, sp = blockIdx.x / p.row_tiles, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gr = lane >> 2, c4 = lane & 3;
  int n_b, held, total;
  if (!kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total)) return;
  const int rows = n_b * p.group;
  if (mt * ROWS >= rows) return;
  const int bh = b * g.hkv + h;
  const long long trow = (long long)bh * g.nb_cap;
  const int t0 = g.next_pos[b];
  const int t_lo = t0 + mt * ROWS / p.group, t_hi = t0 + (min(rows, mt * ROWS + ROWS) - 1) / p.group;
  if (tid < WARPS * ST) mbar_init(&bars[tid / ST][tid % ST], 1);
  if (tid < 3) sm_cnt[tid] = 0;
  if (tid == 0) sm_abort = 0;
  fence_mbar_init();
  __syncthreads();

  const int nb = (total + g.tile - 1) / g.tile;
  const KvRange rg = kv_range(g, p, trow, nb, t_lo, t_hi, t0 + n_b - 1, sm_cnt, tid, WARPS * 32);
  const int ppt = g.tile / PIECE;
  // pieces behind the last token, where its tile is among them
  const int tail = rg.upto == nb && (rg.from < nb || rg.n_first == nb) ? (nb * g.tile - total) / PIECE : 0;
  const int pieces = max(0, rg.count() * ppt - tail);
  const int per = (pieces + p.splits - 1) / p.splits;
  const int p_lo = sp * per, p_hi = min(pieces, p_lo + per);
  const int mine = p_hi - p_lo > warp ? (p_hi - p_lo - warp + WARPS - 1) / WARPS : 0;  // this warp's pieces
  // place of the warp's k-th piece: its tile's entry, and which part of the tile
  auto place = [&](int k, int& sub) {
    const int pc = p_lo + warp + k * WARPS, vt = pc / ppt;
    sub = pc - vt * ppt;
    return rg.tile(vt);
  };
  uint8_t* ring = smem + warp * ST * 2 * Cfg::PB;
  int row_of = 0;  // lane j: pool row of the piece issued (32-blockwise) j-th, -1 for none
  auto issue = [&](int k) {
    if ((k & 31) == 0) {
      row_of = -1;
      if (k + lane < mine) {
        int sub;
        const int i = place(k + lane, sub);
        const int slot = g.table[trow + i];
        if (slot >= 0 && slot < g.n_slots) row_of = slot * g.tile + sub * PIECE;
        else report(g.dev_status, VEDA_ERR_BAD_INDEX);
      }
    }
    const int row = __shfl_sync(0xffffffffu, row_of, k & 31);
    if (lane == 0 && row >= 0) {
      uint64_t* bar = &bars[warp][k % ST];
      uint8_t* dst = ring + (k % ST) * 2 * Cfg::PB;
      mbar_expect_tx(bar, 2 * Cfg::PB);
      tma_load_2d(dst, &maps.k, bar, 0, row);
      tma_load_2d(dst + Cfg::PB, &maps.v, bar, 0, row);
    }
    return row >= 0;
  };
  uint32_t there = 0;  // bit s: stage s holds a piece (not an absent tile)
  int issued = 0;
  for (; issued < ST && issued < mine; ++issued)
    if (issue(issued)) there |= 1u << issued;

  // Q as fp16 fragments, each row times a power of two that puts its largest
  // value into [2^13, 2^14): bf16's range fits, and its 8 bits are kept down
  // to 2^-37 of the row's largest
  const int r0 = mt * ROWS + gr, r1 = r0 + 8;
  uint32_t qa[KS][4];
  float qs[2];
  int tq[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = e ? r1 : r0;
    tq[e] = t0 + r / p.group;
    uint2 w[KS];
    uint32_t top = 0;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      w[ks] = make_uint2(0, 0);
      if (r < rows)
        w[ks] = *reinterpret_cast<const uint2*>(p.q.p + b * p.q.sb + (long long)(r / p.group) * p.q.sn +
                                                (long long)(h * p.group + r % p.group) * p.q.sh + ks * 16 + c4 * 4);
      top = max(top, max(bf16x2_top(w[ks].x), bf16x2_top(w[ks].y)));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    float mul;
    q_scale<13>(top, mul, qs[e]);
    qs[e] *= p.scale_log2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][e] = pack_f16x2(__uint_as_float(w[ks].x << 16) * mul, __uint_as_float(w[ks].x & 0xffff0000u) * mul);
      qa[ks][2 + e] = pack_f16x2(__uint_as_float(w[ks].y << 16) * mul, __uint_as_float(w[ks].y & 0xffff0000u) * mul);
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[KS][2][4];
#pragma unroll
  for (int c = 0; c < KS; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[c][e][x] = 0.f;

  int pos_of = 0;  // lane j: as row_of, for the piece computed j-th
  float sk_of = 0.f, sv_of = 0.f;
  bool ok = true;
  uint32_t phase = 0;  // bit s: parity of stage s
  for (int k = 0; k < mine; ++k) {
    const int st = k % ST;
    int sub;
    const int i = place(k, sub);
    if ((k & 31) == 0 && k + lane < mine) {
      int sb;
      const long long e = trow + place(k + lane, sb);
      pos_of = g.pos[e] + sb * PIECE;
      sk_of = g.k_scale[e];
      sv_of = g.v_scale[e];
    }
    const int pos0 = __shfl_sync(0xffffffffu, pos_of, k & 31);
    const float sk = __shfl_sync(0xffffffffu, sk_of, k & 31), sv = __shfl_sync(0xffffffffu, sv_of, k & 31);
    if (!(there >> st & 1u)) {
      if (p.lw && lane < ROWS && mt * ROWS + lane < rows)
        p.lw[((long long)bh * p.pieces_cap + i * ppt + sub) * p.rows_cap + mt * ROWS + lane] = -INFINITY;
    } else {
    if (!__all_sync(0xffffffffu, mbar_wait(&bars[warp][st], phase >> st & 1u, &sm_abort, g.dev_status))) {
      ok = false;
      break;
    }
    phase ^= 1u << st;
    const uint32_t ka = smem_u32(ring + st * 2 * Cfg::PB), va = ka + Cfg::PB;
    const int left = total - (i * g.tile + sub * PIECE);  // keys of the piece that exist
    if (left < PIECE) {
      // V rows behind the last token become zeroes: their codes may be anything
      for (int x = left * D / 16 + lane; x < Cfg::PB / 16; x += 32)
        *reinterpret_cast<uint4*>(ring + st * 2 * Cfg::PB + Cfg::PB + code_at<D>(x / (D / 16), x % (D / 16))) =
            make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    }
    float s[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
      for (int x = 0; x < 4; ++x) s[nt][x] = 0.f;
#pragma unroll
      for (int q4 = 0; q4 < KS / 4; ++q4) {
        uint32_t f[4];
        ldsm4(f, ka + code_at<D>(nt * 8 + (lane & 7), q4 * 4 + (lane >> 3)));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t b0, b1;
          codes_f16(f[x], b0, b1);
          mma(s[nt], qa[q4 * 4 + x], b0, b1);
        }
      }
    }
    const float ev = log2f(sv), rv = 1.0f / sv;
    const float co[2] = {qs[0] * sk, qs[1] * sk};
    const bool whole = left >= PIECE && kv_seen(pos0 + PIECE - 1, t_lo, p.causal, 0, 0) &&
                       (p.window <= 0 || pos0 + PIECE <= p.sinks || (long long)pos0 > (long long)t_hi - p.window);
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = x >> 1, kk = nt * 8 + c4 * 2 + (x & 1);
        float v = s[nt][x] * co[e] + ev;
        if (!whole && !(kk < left && kv_seen(pos0 + kk, tq[e], p.causal, p.window, p.sinks))) v = -INFINITY;
        s[nt][x] = v;
        over |= v > m[e] + MARGIN;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = m[e];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * e], s[nt][2 * e + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float al = mx == m[e] ? 1.f : fast_exp2(m[e] - mx);
        m[e] = mx;
        l[e] *= al;
#pragma unroll
        for (int c = 0; c < KS; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            o[c][y][2 * e] *= al;
            o[c][y][2 * e + 1] *= al;
          }
      }
    }
    float ls[2] = {0.f, 0.f};
    uint32_t pa[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float base = OFF - (m[e] == -INFINITY ? 0.f : m[e]);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float x0 = fast_exp2(s[nt][2 * e] + base), x1 = fast_exp2(s[nt][2 * e + 1] + base);
        ls[e] += x0 + x1;
        pa[nt >> 1][(nt & 1) * 2 + e] = pack_f16x2(x0, x1);
      }
      // the sum without sv; NaN scales reach the rows that see the tile through P, and no other
      l[e] += ls[e] == 0.f ? 0.f : ls[e] * rv;
    }
    if (p.lw) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = ls[e] + __shfl_xor_sync(0xffffffffu, ls[e], 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const int r = e ? r1 : r0;
        if (c4 == 0 && r < rows)
          p.lw[((long long)bh * p.pieces_cap + i * ppt + sub) * p.rows_cap + r] =
              t == 0.f ? -INFINITY : log2f(t) + (m[e] - OFF - ev);
      }
    }
#pragma unroll
    for (int ch = 0; ch < KS; ++ch) {
      uint32_t f[4], ev_f[4], od_f[4];
      ldsm4_t(f, va + code_at<D>(lane, ch));
#pragma unroll
      for (int x = 0; x < 4; ++x) codes_f16(__byte_perm(f[x], 0, 0x3120), ev_f[x], od_f[x]);
      mma(o[ch][0], pa[0], ev_f[0], ev_f[1]);
      mma(o[ch][1], pa[0], od_f[0], od_f[1]);
      mma(o[ch][0], pa[1], ev_f[2], ev_f[3]);
      mma(o[ch][1], pa[1], od_f[2], od_f[3]);
    }
    }
    if (issued < mine) {
      __syncwarp();  // every lane has read the stage
      there = issue(issued) ? there | 1u << st : there & ~(1u << st);
      ++issued;
    }
  }
  if (!ok)  // let every copy that was started land
    for (int s = 0; s < ST; ++s)
      if (there >> s & 1u) mbar_wait_drain(&bars[warp][s], phase >> s & 1u, VEDA_WAIT_LIMIT_NS);

  // join the warps: references, then sums and O in warp order
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    if (c4 == 0) sm_m[warp][gr + 8 * e] = m[e];
  }
  __syncthreads();
  float* acc = reinterpret_cast<float*>(smem);  // [WARPS][ROWS][D], in the ring
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float mx = sm_m[0][gr + 8 * e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, sm_m[w][gr + 8 * e]);
    const float f = m[e] == -INFINITY ? (l[e] == l[e] ? 0.f : 1.f) : fast_exp2(m[e] - mx);
    if (c4 == 0) sm_l[warp][gr + 8 * e] = l[e] * f;
#pragma unroll
    for (int ch = 0; ch < KS; ++ch)
      *reinterpret_cast<float4*>(acc + (warp * ROWS + gr + 8 * e) * D + ch * 16 + c4 * 4) = make_float4(
          o[ch][0][2 * e] * f, o[ch][1][2 * e] * f, o[ch][0][2 * e + 1] * f, o[ch][1][2 * e + 1] * f);
  }
  __syncthreads();
  const long long prow = ((long long)bh * p.splits + sp) * p.rows_pad + mt * ROWS;
  for (int x = tid; x < ROWS * D / 4; x += WARPS * 32) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    if (mt * ROWS + r >= rows) break;
    float4 v = *reinterpret_cast<float4*>(acc + r * D + c);
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float4 u = *reinterpret_cast<float4*>(acc + (w * ROWS + r) * D + c);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    *reinterpret_cast<float4*>(p.part_o + (prow + r) * D + c) = v;
  }
  if (tid < ROWS) {
    float lsum = 0.f, mm = sm_m[0][tid];
    for (int w = 0; w < WARPS; ++w) {
      lsum += sm_l[w][tid];
      mm = fmaxf(mm, sm_m[w][tid]);
    }
    p.part_ml[prow + tid] = make_float2(mm, lsum);
  }
}

// Joins the splits of a row: a warp per row.
template <int D>
__global__ void __launch_bounds__(128) kv_join_kernel(const KvGeom g, const KvAttnParams p) {
  const int lane = threadIdx.x % 32, h = blockIdx.y, b = blockIdx.z;
  const int r = blockIdx.x * 4 + threadIdx.x / 32;
  int n_b, held, total;
  if (!kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total)) return;
  if (r >= n_b * p.group) return;
  const int bh = b * g.hkv + h;
  const long long rows = p.rows_pad;
  const float2* ml = p.part_ml + (long long)bh * p.splits * rows + r;
  float m = -INFINITY;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, ml[s * rows].x);
  float l = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 x = ml[s * rows];
    const float f = x.x == -INFINITY ? (x.y == x.y ? 0.f : 1.f) : fast_exp2(x.x - m);
    l += x.y * f;
    const float* src = p.part_o + (((long long)bh * p.splits + s) * rows + r) * D + lane * (D / 32);
    if constexpr (D == 128) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      o[0] += v.x * f;
      o[1] += v.y * f;
      o[2] += v.z * f;
      o[3] += v.w * f;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      o[0] += v.x * f;
      o[1] += v.y * f;
    }
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.0f / l;
  const int i = r / p.group, qh = h * p.group + r % p.group;
  __nv_bfloat16* dst = p.o + b * p.o_sb + (long long)i * p.o_sn + (long long)qh * p.o_sh + lane * (D / 32);
  uint32_t w[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) w[e] = pack_bf16x2_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) reinterpret_cast<uint32_t*>(dst)[e] = w[e];
  if (lane == 0) {
    const float l2 = none ? -INFINITY : log2f(l) + (m == -INFINITY ? 0.f : m) - OFF;
    if (p.lse) p.lse[((long long)b * p.heads + qh) * p.n_q + i] = l2 * LN2;
    if (p.lse2) p.lse2[(long long)bh * p.rows_cap + r] = l2;
  }
}

// weight[tile] = decay * weight[tile] + sum over rows and the tile's pieces of
// 2^(lw - lse2): a block per tile, its sums joined in a fixed order.
constexpr int WEIGHT_THREADS = 256;  // a row tile's rows at most
__global__ void __launch_bounds__(WEIGHT_THREADS) kv_weight_kernel(const KvGeom g, const KvAttnParams p) {
  __shared__ float part[WEIGHT_THREADS / 32];
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int n_b, held, total;
  if (!kv_counts(g, b, h, p.n_q, p.n_new, p.pending, n_b, held, total)) return;
  const int nb = (total + g.tile - 1) / g.tile;
  if (i >= nb || n_b == 0) return;
  const int bh = b * g.hkv + h, ppt = g.tile / p.piece;
  const long long entry = (long long)bh * g.nb_cap + i;
  const int rows = n_b * p.group, t0 = g.next_pos[b], ps = g.pos[entry];
  const float* lse2 = p.lse2 + (long long)bh * p.rows_cap;
  const float* lw = p.lw + ((long long)bh * p.pieces_cap + (long long)i * ppt) * p.rows_cap;
  float w = 0.f;
  // row tile by row tile: only tiles that a row tile's CTA could see were visited
#pragma unroll 4
  for (int m0 = 0; m0 < rows; m0 += p.tile_rows) {
    const int m1 = min(rows, m0 + p.tile_rows) - 1, r = m0 + tid;
    if (r > m1 || !kv_tile_seen(ps, g.tile, t0 + m0 / p.group, t0 + m1 / p.group, p.causal, p.window, p.sinks)) continue;
    const float z = lse2[r];
    if (z == -INFINITY) continue;
    for (int k = 0; k < ppt && i * g.tile + k * p.piece < total; ++k) {
      const float x = lw[(long long)k * p.rows_cap + r];
      if (x != -INFINITY) w += fast_exp2(x - z);  // none of it seen: nothing, even of a row that is NaN
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
  if (tid % 32 == 0) part[tid / 32] = w;
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < WEIGHT_THREADS / 32; ++k) w += part[k];
    p.weight[entry] = p.decay == 0.f ? w : p.decay * p.weight[entry] + w;
  }
}

template <int D>
cudaError_t launch_rows(const KvGeom& g, const KvAttnParams& p, cudaStream_t s) {
  KvMaps maps;
  const uint64_t rows = (uint64_t)g.n_slots * g.tile;
  if (encode_tensor_map_2d_u8(&maps.k, g.k8, D, rows, PIECE) != CUDA_SUCCESS ||
      encode_tensor_map_2d_u8(&maps.v, g.v8, D, rows, PIECE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e =
      cudaFuncSetAttribute(kv_attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  kv_attn_rows_kernel<D><<<dim3(p.row_tiles * p.splits, g.hkv, g.B), WARPS * 32, RowsCfg<D>::SMEM, s>>>(g, p, maps);
  return cudaGetLastError();
}

}  // namespace

// Tokens that the rows of a row tile span.
static int n_tok(int rows, int group) { return (rows + group - 1) / group + 1; }

size_t kv_attn_plan(const KvGeom& g, KvAttnParams& p, bool weights, uint8_t* ws) {
  const long long rows = (long long)p.n_q * p.group;
  p.tiles = rows > TILE_KERNEL_ROWS;
  p.tile_rows = p.tiles ? 256 : ROWS;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  p.rows_cap = (int)rows;
  p.rows_pad = p.row_tiles * p.tile_rows;
  p.piece = p.tiles ? g.tile : PIECE;
  p.pieces_cap = g.nb_cap * (g.tile / p.piece);
  const long long ctas = (long long)g.B * g.hkv * p.row_tiles, keys = (long long)g.nb_cap * g.tile;
  p.splits = 1;
  if (p.tiles) {
    // One CTA per SM: waves of CTAs, each as long as its steps and what begins
    // and ends it; what is split is written and read once more and joined.
    // Measured at d = 128: 2.1 us a step, 5 us a CTA, 8 us for the join.
    const long long see = p.window > 0 ? (long long)p.window + p.sinks + n_tok(p.tile_rows, p.group) + 2 * g.tile : keys;
    const double steps = (double)((see < keys ? see : keys) + 127) / 128, t = 2.1 * g.d / 128;
    double best = 0;
    for (int s = 1; s <= 32 && (s == 1 || steps >= 3 * s); ++s) {
      const double waves = (double)((ctas * s + 147) / 148);
      const double us = waves * (ceil(steps / s) * t + 5) +
                        (s > 1 ? 8 + (double)ctas * s * p.tile_rows * g.d * 8 / 4e6 : 0);
      if (s == 1 || us < best) {
        best = us;
        p.splits = s;
      }
    }
  } else {
    const long long want = (148 * 6 + ctas - 1) / ctas, most = (keys + PIECE * WARPS - 1) / (PIECE * WARPS);
    p.splits = (int)(want < most ? want : most);
    if (p.splits < 1) p.splits = 1;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = ws ? ws + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t prows = (size_t)g.B * g.hkv * p.splits * p.rows_pad;
  p.part_ml = reinterpret_cast<float2*>(take(prows * 8));
  p.part_o = p.tiles && p.splits == 1 ? nullptr : reinterpret_cast<float*>(take(prows * g.d * 4));
  p.lse2 = nullptr;
  p.lw = nullptr;
  if (weights) {
    p.lse2 = reinterpret_cast<float*>(take((size_t)g.B * g.hkv * rows * 4));
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
  cudaError_t e = p.tiles ? launch_kv_attn_tiles(g, p, s) : g.d == 128 ? launch_rows<128>(g, p, s) : launch_rows<64>(g, p, s);
  if (e != cudaSuccess) return e;
  if (!p.tiles || p.splits > 1) {
    const dim3 jg((p.rows_cap + 3) / 4, g.hkv, g.B);
    if (g.d == 128) kv_join_kernel<128><<<jg, 128, 0, s>>>(g, p);
    else kv_join_kernel<64><<<jg, 128, 0, s>>>(g, p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !p.weight) return e;
  kv_weight_kernel<<<dim3(g.nb_cap, g.hkv, g.B), WEIGHT_THREADS, 0, s>>>(g, p);
  return cudaGetLastError();
}

}  // namespace veda
