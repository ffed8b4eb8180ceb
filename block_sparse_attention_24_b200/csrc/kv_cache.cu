// The 8-bit K/V tile cache: writing new tokens into it (append), taking them
// in (advance) and dropping its least used tiles (evict).
//
// A cached value is code * scale with an e4m3 code and one scale per (sequence,
// K/V head, tile), separate for K and V. The scale is a power of two, so that
// dividing by it, changing it later and folding it into an exponent are exact;
// a floating-point code loses no precision by that, only range, of which 448
// to 2^-9 leaves plenty.
#include "kv_attn.cuh"

namespace veda {
namespace {

constexpr int APPEND_THREADS = 256;
static_assert(APPEND_THREADS >= VEDA_MAX_HEADS, "a thread looks at each head's count");

// The least power of two s with 448 s >= a (a >= 0), at least 2^-40; NaN
// where a is not finite or s would pass 2^80. 448 = 1.75 * 2^8, so the
// exponent is that of a, less 8, and one more where a's significand passes
// 1.75.
__device__ __forceinline__ float scale_of(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < -40) e = -40;
  if (u >= 0x7f800000u || e > 80) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float2 unpack_e4m3x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The codes of four bf16 values times f, and of four codes times f.
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, float f) {
  return pack_e4m3x4(bf_lo(a) * f, bf_hi(a) * f, bf_lo(b) * f, bf_hi(b) * f);
}
__device__ __forceinline__ uint32_t codes_moved(uint32_t c, float f) {
  const float2 a = unpack_e4m3x2((uint16_t)c), b = unpack_e4m3x2((uint16_t)(c >> 16));
  return pack_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ uint4 codes_moved(uint4 w, float f) {
  return make_uint4(codes_moved(w.x, f), codes_moved(w.y, f), codes_moved(w.z, f), codes_moved(w.w, f));
}

// One tile of K or of V of one head: scale' = max(old scale, the new tokens'),
// old codes moved to it (rounded once more where it grew), new ones quantised,
// the rows behind the last token zeroed. The tile's bf16 rows are held in
// registers between the maximum and the rounding, so they are read once:
// 2 bytes in and 1 out per value. 3,840 tokens of 24 heads, d = 128: 14.9 us,
// 4.7 TB/s (of 6.5 measured for a copy). In earlier forms of this kernel five to
// seven CTAs per SM instead of four, by fewer registers, took 16.5 to 22.3 us
// where four took 16.6, and 128 or 512 threads 19 where 256 took 15.1.
//
// The older codes of a tile that tokens join are rounded in place, and those
// tokens are only pending: the codes and the scale as they were go to `tail`
// (by the one CTA that has this tile), and the next append starts from them. It
// knows them to be the tile's by the slot, the row count and next_pos, all as
// they were, and by the scale and codes there, which must be what the raise
// left: otherwise tokens were taken in since, or put there by the caller.
template <int D>
__global__ void __launch_bounds__(APPEND_THREADS)
    kv_append_kernel(const KvGeom g, const KvTail tail, const KvRows kr, const KvRows vr, const int n,
                     const int32_t* n_new) {
  constexpr int VPR = D / 16;                          // 16-value vectors per row
  constexpr int PT = 128 * VPR / APPEND_THREADS;       // vectors per thread at tile 128
  const int h = blockIdx.y >> 1, is_v = blockIdx.y & 1, b = blockIdx.z;
  after_predecessor();
  // kv_counts, but for the other heads, whose counts are looked at where the
  // block meets, while rows are on their way (before them: frame 15.1 us, not 14.9)
  const int32_t* len = g.len + (long long)b * g.hkv;
  const int other = threadIdx.x < g.hkv ? len[threadIdx.x] : 0;
  const int held = len[h], n_b = n_new ? n_new[b] : n;
  const long long room = (long long)g.nb_cap * g.tile - n_b;
  if (n_b < 0 || n_b > n || held < 0 || held > room) {
    report(g.dev_status, VEDA_ERR_BAD_INDEX);
    return;
  }
  const int i = held / g.tile + blockIdx.x;            // the tile's place in the table
  const int row0 = i * g.tile - held;                  // new token in its first row (negative: that row is older)
  const bool fresh = row0 >= 0, first = blockIdx.x == 0 && tail.codes;
  const long long kept = ((long long)b * g.hkv + h) * 2 + is_v;
  if (n_b == 0 ? !first || fresh : row0 >= n_b) return;
  const long long entry = ((long long)b * g.hkv + h) * g.nb_cap + i;
  float* scale = (is_v ? g.v_scale : g.k_scale) + entry;
  const KvRows& x = is_v ? vr : kr;
  const __nv_bfloat16* src = x.p + b * x.sb + h * x.sh;
  // in flight with the rows
  const int slot = g.table[entry];
  float s_old = fresh ? 0.f : *scale;
  const bool joins = first && !fresh;
  const int4 key = joins ? tail.key[kept] : make_int4(0, 0, 0, 0);
  const float2 was = joins ? tail.scale[kept] : make_float2(0.f, 0.f);
  const int next = joins ? g.next_pos[b] : 0;

  uint4 val[PT][2];
#pragma unroll
  for (int j = 0; j < PT; ++j) {
    const int vec = threadIdx.x + j * APPEND_THREADS, r = vec / VPR, c = vec % VPR, t = row0 + r;
    val[j][0] = val[j][1] = make_uint4(0, 0, 0, 0);
    if (r < g.tile && t >= 0 && t < n_b) {
      const uint4* q = reinterpret_cast<const uint4*>(src + (long long)t * x.sn + c * 16);
      val[j][0] = __ldcs(q);  // read once
      val[j][1] = __ldcs(q + 1);
    }
  }
  const bool absent = slot < 0 || slot >= g.n_slots;
  uint8_t* codes = (is_v ? g.v8 : g.k8) + (long long)slot * g.tile * D;
  uint8_t* const kept_codes = tail.codes + kept * g.tile * D;
  // the tail may be what a raise left of the kept codes: both are looked at, in
  // the registers of the rows that are not new (in a loop and registers of their
  // own the frame took 15.5 us where it took 14.7, one token 4.3 where it took 3.5)
  const bool raise_left = joins && !absent && key.x == -row0 && key.y == slot && key.z == next &&
                          __float_as_uint(was.y) == __float_as_uint(s_old);
  bool back = raise_left;  // the kept codes and scale are the committed ones
  if (raise_left) {
    const float f = was.x * (1.0f / was.y);
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int vec = threadIdx.x + j * APPEND_THREADS;
      if (vec < -row0 * VPR) {
        val[j][0] = reinterpret_cast<const uint4*>(codes)[vec];
        val[j][1] = reinterpret_cast<const uint4*>(kept_codes)[vec];
      }
    }
#pragma unroll
    for (int j = 0; j < PT; ++j)
      if (threadIdx.x + j * APPEND_THREADS < -row0 * VPR) {
        const uint4 w = val[j][0], m = was.y == was.y ? codes_moved(val[j][1], f) : val[j][1];
        back = back && w.x == m.x && w.y == m.y && w.z == m.z && w.w == m.w;
      }
  }
  // the largest |x| by its bits: infinities and NaN come out above every finite value
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < PT; ++j)
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (fresh || threadIdx.x + j * APPEND_THREADS >= -row0 * VPR)  // (older rows: codes, or nothing)
        top = max(top, max(max(bf16x2_top(val[j][y].x), bf16x2_top(val[j][y].y)),
                           max(bf16x2_top(val[j][y].z), bf16x2_top(val[j][y].w))));
  __shared__ uint32_t warp_top[APPEND_THREADS / 32];
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) warp_top[threadIdx.x / 32] = top;
  if (__syncthreads_or(other < 0 || other > room)) {
    if (threadIdx.x == 0) report(g.dev_status, VEDA_ERR_BAD_INDEX);
    return;
  }
  if (raise_left) {
    back = __syncthreads_and(back);
    if (back) s_old = was.x;
  }
#pragma unroll
  for (int w = 0; w < APPEND_THREADS / 32; ++w) top = max(top, warp_top[w]);
  if (n_b == 0 && !back) return;
  if (absent) {  // no codes, but a place in the stream like any tile
    if (threadIdx.x == 0) {
      report(g.dev_status, VEDA_ERR_BAD_INDEX);
      if (fresh && !is_v) g.pos[entry] = g.next_pos[b] + row0;
    }
    return;
  }
  const float s_new = scale_of(__uint_as_float(top));
  float s = fresh ? s_new : ((s_new != s_new || s_old != s_old) ? s_new + s_old : fmaxf(s_new, s_old));
  if (n_b == 0) s = s_old;
  const bool fine = s == s;
  const float inv = fine ? 1.0f / s : 0.f;
  const bool raised = !fresh && s_old == s_old && s != s_old;

#pragma unroll
  for (int j = 0; j < PT; ++j) {
    const int vec = threadIdx.x + j * APPEND_THREADS, r = vec / VPR, c = vec % VPR, t = row0 + r;
    if (r >= g.tile) continue;
    uint4* dst = reinterpret_cast<uint4*>(codes + r * D + c * 16);
    if (t >= 0) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (t < n_b && fine) {
        const uint4 a = val[j][0], e = val[j][1];
        o = make_uint4(codes_of(a.x, a.y, inv), codes_of(a.z, a.w, inv), codes_of(e.x, e.y, inv), codes_of(e.z, e.w, inv));
      }
      *dst = o;
    } else if (raised || back) {
      uint4 w = back ? val[j][1] : *dst;
      if (raised && first && !back) *reinterpret_cast<uint4*>(kept_codes + r * D + c * 16) = w;
      if (raised && fine) w = codes_moved(w, s_old * inv);
      *dst = w;
    }
  }
  if (threadIdx.x == 0) {
    *scale = s;
    if (first) {
      tail.key[kept] = raised ? make_int4(-row0, slot, next, 0) : make_int4(0, 0, 0, 0);
      if (raised) tail.scale[kept] = make_float2(s_old, s);
    }
    if (fresh && !is_v) {
      g.pos[entry] = g.next_pos[b] + row0;
      if (g.weight) g.weight[entry] = 0.f;
    }
  }
}

// A warp per sequence.
__global__ void kv_advance_kernel(const KvGeom g, const int n, const int32_t* n_new) {
  after_predecessor();
  const int b = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
  if (b >= g.B) return;
  int n_b, held, total;
  if (!kv_counts(g, b, 0, n, n_new, true, n_b, held, total)) return;
  for (int h = lane; h < g.hkv; h += 32) g.len[(long long)b * g.hkv + h] += n_b;
  if (lane == 0) g.next_pos[b] += n_b;
}

struct KvKeep {
  int32_t k[VEDA_MAX_HEADS];
};

// fp32 bits -> unsigned keys that rank as the values do; -0 as +0, NaN first.
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of `flag` over the block, and its total.
template <int THREADS>
__device__ __forceinline__ int block_prefix(bool flag, int* warp_n, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();  // the last call's counts have been read
  if (lane == 0) warp_n[warp] = __popc(m);
  __syncthreads();
  // every warp sums the counts for itself
  const int c = lane < THREADS / 32 ? warp_n[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, c);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
  return before + __popc(m & ((1u << lane) - 1u));
}

// One (sequence, head): the row of the table is read whole into shared
// memory, the weight of the last tile that stays is found by radix selection
// (8 bits at a time; weights mostly share their exponents, so eight
// histograms, by lane, keep the counters apart), and the row is written back
// with the tiles that stay first, in their order, then those that go, then the
// free ones. Nothing of the codes moves. Latency, not bandwidth, is the bound,
// so the block has a thread per entry or few (eight at most): 24 rows of 300
// entries take 5.6 us, 256 rows of 2,047 take 9.4 us.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    kv_evict_kernel(const KvGeom g, const KvGeom out, const KvKeep keeps, const int sink, const int recent) {
  extern __shared__ uint32_t sm[];
  const int cap = (g.nb_cap + 3) & ~3;
  uint32_t* f_table = sm;
  uint32_t* f_pos = sm + cap;
  uint32_t* f_ks = sm + 2 * cap;
  uint32_t* f_vs = sm + 3 * cap;
  uint32_t* f_w = sm + 4 * cap;
  __shared__ int hist[8][256];
  __shared__ int warp_n[32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_want, sh_found;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid % 32;
  const int bh = b * g.hkv + h;
  const long long row = (long long)bh * g.nb_cap;
  after_predecessor();
  const int held = g.len[bh];
  const bool same = out.table == g.table;
  // a row starts at a multiple of 16 bytes where its length is one of 4
  if (g.nb_cap % 4 == 0) {
    for (int i = tid; i < g.nb_cap / 4; i += THREADS) {
      reinterpret_cast<uint4*>(f_table)[i] = reinterpret_cast<const uint4*>(g.table + row)[i];
      reinterpret_cast<uint4*>(f_pos)[i] = reinterpret_cast<const uint4*>(g.pos + row)[i];
      reinterpret_cast<uint4*>(f_ks)[i] = reinterpret_cast<const uint4*>(g.k_scale + row)[i];
      reinterpret_cast<uint4*>(f_vs)[i] = reinterpret_cast<const uint4*>(g.v_scale + row)[i];
      reinterpret_cast<uint4*>(f_w)[i] = reinterpret_cast<const uint4*>(g.weight + row)[i];
    }
  } else {
#pragma unroll 2
    for (int i = tid; i < g.nb_cap; i += THREADS) {
      const uint32_t a = (uint32_t)g.table[row + i], c = (uint32_t)g.pos[row + i], d = __float_as_uint(g.k_scale[row + i]),
                     e = __float_as_uint(g.v_scale[row + i]), f = __float_as_uint(g.weight[row + i]);
      f_table[i] = a;
      f_pos[i] = c;
      f_ks[i] = d;
      f_vs[i] = e;
      f_w[i] = f;
    }
  }
  const bool bad = held < 0 || (long long)held > (long long)g.nb_cap * g.tile;
  if (bad && tid == 0) report(g.dev_status, VEDA_ERR_BAD_INDEX);
  const int nb = bad ? 0 : (int)(((long long)held + g.tile - 1) / g.tile);
  const int keep = keeps.k[h];
  const bool cut = nb > keep;
  if (!cut && same) return;
  for (int i = tid; i < 8 * 256; i += THREADS) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto put = [&](int i, int to) {
    out.table[row + to] = (int32_t)f_table[i];
    out.pos[row + to] = (int32_t)f_pos[i];
    out.k_scale[row + to] = __uint_as_float(f_ks[i]);
    out.v_scale[row + to] = __uint_as_float(f_vs[i]);
    out.weight[row + to] = __uint_as_float(f_w[i]);
  };
  if (h == 0 && tid == 0 && !same) out.next_pos[b] = g.next_pos[b];
  if (!cut) {
    for (int i = tid; i < g.nb_cap; i += THREADS) put(i, i);
    if (tid == 0) out.len[bh] = held;
    return;
  }
  // the key of the last tile that stays among [sink, nb - recent), and how
  // many with exactly that key stay
  const int lo = sink, hi = nb - recent;
  int want = keep - sink - recent;
  const bool none = want == 0;
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0 && !none; shift -= 8) {
    for (int i = lo + tid; i < hi; i += THREADS) {
      const uint32_t k = rank_key(__uint_as_float(f_w[i]));
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[lane & 7][(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid < 256) {  // thread t has bin 255 - t, so that a prefix counts from the top
      int c = 0;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        c += hist[y][255 - tid];
        hist[y][255 - tid] = 0;
      }
      int incl = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (lane == 31) warp_n[tid / 32] = incl;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int w = lane < 8 ? warp_n[lane] : 0;
      const int above = __reduce_add_sync(0xffffffffu, lane < tid / 32 ? w : 0) + incl - c;
      if (above < want && want <= above + c) {
        sh_prefix = prefix | ((uint32_t)(255 - tid) << shift);
        sh_want = want - above;
        sh_found = c;
      }
    }
    __syncthreads();
    prefix = sh_prefix;
    want = sh_want;
  }
  // where all that share the last key stay, none of them has to be counted
  const bool all = none || sh_found == want;
  int stays = 0, goes = 0, ties = 0;
  for (int base = 0; base < nb; base += THREADS) {
    const int i = base + tid;
    const bool mid = i >= lo && i < hi, in = i < nb;
    const uint32_t k = mid ? rank_key(__uint_as_float(f_w[i])) : 0;
    const bool tie = mid && !none && k == prefix;
    int n_tie = 0, n_stay, t = 0;
    if (!all) t = block_prefix<THREADS>(tie, warp_n, n_tie);
    const bool stay = in && (!mid || (!none && (k > prefix || (tie && (all || ties + t < want)))));
    const int r = block_prefix<THREADS>(stay, warp_n, n_stay);
    if (in) put(i, stay ? stays + r : keep + goes + (tid - r));
    ties += n_tie;
    stays += n_stay;
    goes += min(THREADS, nb - base) - n_stay;
  }
  if (!same)
    for (int i = nb + tid; i < g.nb_cap; i += THREADS) put(i, i);
  if (tid == 0) out.len[bh] = held - (nb - keep) * g.tile;
}

template <int THREADS>
cudaError_t launch_evict(const KvGeom& g, const KvKeep& keeps, int sink, int recent, const KvGeom& out, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const int smem = 5 * 4 * ((g.nb_cap + 3) & ~3);
  const cudaError_t e = allow_smem((const void*)kv_evict_kernel<THREADS>, 5 * 4 * VEDA_KV_MAX_NB, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kv_evict_kernel<THREADS>, dim3(g.hkv, g.B), THREADS, smem, s, g, out, keeps, sink, recent);
}

}  // namespace

cudaError_t launch_kv_append(const KvGeom& g, const KvTail& tail, const KvRows& k, const KvRows& v, int n,
                             const int32_t* n_new, cudaStream_t s) {
  const long long tiles = ((long long)n + g.tile - 2) / g.tile + 1;  // n tokens from any row of a tile on
  const dim3 grid((unsigned)(tiles < g.nb_cap ? tiles : g.nb_cap), 2 * g.hkv, g.B);
  return launch_chained(g.d == 128 ? kv_append_kernel<128> : kv_append_kernel<64>, grid, APPEND_THREADS, 0, s, g, tail, k,
                        v, n, n_new);
}

cudaError_t launch_kv_advance(const KvGeom& g, int n, const int32_t* n_new, cudaStream_t s) {
  return launch_chained(kv_advance_kernel, dim3((g.B + 3) / 4), 128, 0, s, g, n, n_new);
}

cudaError_t launch_kv_evict(const KvGeom& g, const int32_t* keep, int sink, int recent, const KvGeom& out,
                            cudaStream_t s) {
  KvKeep keeps;
  for (int h = 0; h < g.hkv; ++h) keeps.k[h] = keep[h];
  return g.nb_cap <= 1024 ? launch_evict<256>(g, keeps, sink, recent, out, s)
                          : g.nb_cap <= 2048 ? launch_evict<512>(g, keeps, sink, recent, out, s)
                                             : launch_evict<1024>(g, keeps, sink, recent, out, s);
}

}  // namespace veda
