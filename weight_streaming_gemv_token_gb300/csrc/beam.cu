// beam_select and beam_reorder_pages: beam search's selection over beams and
// vocabulary, and the page tables and tail pages of the beams it leaves.
//
// Selection. A candidate (b, v) has the key score_b + (x_bv - lse_b), lse_b =
// log sum exp x_b. Every logit is read once from memory:
//   pass 1  one CTA per chunk of a row: the chunk's maximum (with its lowest
//           index) and sum of exp(x - maximum), the running pair of a softmax;
//   pass 2  every CTA joins the chunks' pairs into the rows' lse, so that each
//           chunk's maximum becomes a key. The n_out-th best of these keys (by
//           histograms) is a lower bound T of the n_out-th best candidate, and only
//           the at most n_out chunks whose maximum reaches T hold selected ones. CTA i
//           re-reads the i-th of them (from L2) and lists the candidates that
//           reach T; the last CTA to finish narrows the
//           listed ones to n_out in the same way, where they are many, and ranks them.
// Candidates are ordered by (key descending, flat index ascending), a total order of
// the keys as the kernels have them (48 bits, lse over a float32 sum): among those T is
// exact, ties included, and the result does not depend on timing. Candidates of different
// beams whose exact keys lie closer than the sums' rounding (about 1e-6) may change places.
// Measured: 4 beams x 151,936 12 us, 64 beams 23 us, of which pass 1 takes 4 and
// 10 (3.9 TB/s) and pass 2 a chain of barriers and L2 round trips.
// Many candidates at the bar (equal or sorted logits, fewer chunks than outputs) are
// narrowed by that one CTA: 4 beams of 151,936 equal logits, 64 outputs 500 us; sorted
// ones 86.
#include <cfloat>
#include <cmath>

#include "beam_plan.h"
#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kChunkCtas = 4;  // CTAs of pass 1 an SM: registers and threads for one of pass 2 remain
constexpr int kBeamRank = 512;     // candidates ranked against each other without narrowing
constexpr int kBeamsMax = 1024, kBeamOutMax = 1024;
constexpr size_t kBeamSmem = 12 * kBeamGather;  // dynamic shared memory of pass 2
static_assert(kBeamChunksMax <= kBeamGather, "the chunks' keys lie where the candidates do");

struct BeamArgs {
  int beams, vocab, n_out, chunk, per_row, chunks, slots, list;
  const float* logits;
  long long stride;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  float4* part;  // of the chunks: maximum, sum, index bits
  uint32_t *counter, *count, *flat;
  uint2* key;  // (high word, low word)
  unsigned long long row_inv;  // k * row_inv >> 32 = k / per_row for a chunk k
  int vec;
  int row_lanes;  // log2 of the lanes that join a row in pass 2
};

// Masked logits (NaN as well) count as -inf.
__device__ __forceinline__ float masked(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A float as an integer in the same order (0 only for a NaN), and back.
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unorder32(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }

// Two floats that sum to a + b exactly.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return make_float2(s, (a - (s - t)) + (b - t));
}

// The key x + off + rest as two order words, the sum as two floats (value and remainder,
// 48 bits): the slow double pipe takes 7 times as long here.
__device__ __forceinline__ uint2 key_words(float x, float2 off, float rest) {
  const float2 s = two_sum(x, off.x), e = two_sum(s.y, off.y);
  // below the lowest finite value: that value, behind those that reach it (fmaxf drops a NaN)
  const float hi = fmaxf(s.x + e.x, -FLT_MAX), lo = fmaxf(e.x - (hi - s.x) + (e.y + rest), -INFINITY);
  return make_uint2(order32(hi), order32(lo));
}

// (score - log s) - m as three floats, the last one `rest`; the bracket is rounded to two
// first, so that rows of one score and sum have the same key at their maxima whatever m is
// (float32's lowest value takes the first float for itself). s = 2^e f with f in [0.7,
// 1.42]; log f = 2 artanh u, u = (f - 1) / (f + 1), |u| < 0.172, by its series to u^9 (the
// next term is below 7e-10; the whole is good to 3e-8); e log 2 is an exact product by the
// first 13 bits of log 2 and a small rest.
__device__ __forceinline__ float2 row_offset(float score, float m, float s, float* rest) {
  int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;  // (s >= 1)
  float f = __uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u);
  if (f > 1.41421356f) f *= 0.5f, ++e;
  const float u = __fdividef(f - 1.f, f + 1.f), u2 = u * u;
  const float log_f = 2.f * fmaf(u * u2, fmaf(u2, fmaf(u2, fmaf(u2, 1.f / 9.f, 1.f / 7.f), 1.f / 5.f), 1.f / 3.f), u);
  const float2 l = two_sum(e * -0.693145751953125f, -log_f), n = two_sum(score, l.x);
  const float2 k = two_sum(n.x, n.y + (l.y - e * 1.428606820309417e-6f));
  const float2 d = two_sum(k.x, -m), r = two_sum(d.y, k.y);
  *rest = r.y;
  return make_float2(d.x, r.x);
}

// Pass 1: chunks blockIdx.x, blockIdx.x + gridDim.x, ..., 16 logits a thread at a
// time. The exponentials are 2^((x - m) log2 e) with m the warp's maximum so far.
// Every CTA is resident from the start and leaves room beside it for one of pass
// 2, which gets ready meanwhile.
__global__ void __launch_bounds__(kChunkThreads, 6) beam_chunks_kernel(const BeamArgs a) {
  constexpr int kWarps = kChunkThreads / 32;
  constexpr float kLog2e = 1.44269504088896340736f;
  __shared__ float s_m[2][kWarps], s_s[2][kWarps];
  __shared__ uint32_t s_i[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  if (tid == 0 && blockIdx.x == 0) *a.counter = 0;
  int turn = 0;
  for (int k = blockIdx.x; k < a.chunks; k += gridDim.x, turn ^= 1) {
    const int b = static_cast<int>((k * a.row_inv) >> 32), v0 = (k - b * a.per_row) * a.chunk, n = min(a.chunk, a.vocab - v0);
    const float* x = a.logits + a.stride * b + v0;
    float m = -INFINITY, s = 0.f;  // the warp's maximum, this thread's sum relative to it
    float own = -INFINITY;         // this thread's maximum, first found at `at`
    uint32_t at = 0xffffffffu;
    for (int w0 = warp * 128; w0 < n; w0 += kChunkThreads * 16) {
      float y[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = w0 + lane * 4 + q * kChunkThreads * 4;
        if (a.vec && i + 4 <= n) {
          const float4 f = *reinterpret_cast<const float4*>(x + i);
          y[4 * q] = f.x, y[4 * q + 1] = f.y, y[4 * q + 2] = f.z, y[4 * q + 3] = f.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[4 * q + e] = i + e < n ? x[i + e] : -INFINITY;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = masked(y[e]), top = fmaxf(top, y[e]);
      if (top > own) {
        own = top;
#pragma unroll
        for (int e = 15; e >= 0; --e)
          if (y[e] == top) at = w0 + lane * 4 + (e >> 2) * kChunkThreads * 4 + (e & 3);
      }
      const float m2 = fmaxf(m, warp_max(top));
      if (m2 > -INFINITY) {
        s *= ex2((m - m2) * kLog2e);  // 0 in the first round
        m = m2;
        // (the difference first: m log2 e overflows for the type's lowest values)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += ex2((y[e] - m) * kLog2e);
      }
    }
    s = warp_sum(s);
    at = __reduce_min_sync(0xffffffffu, own == m ? at : 0xffffffffu);
    if (lane == 0) s_m[turn][warp] = m, s_s[turn][warp] = s, s_i[turn][warp] = at;
    __syncthreads();
    if (warp == 0) {
      const float wm = lane < kWarps ? s_m[turn][lane] : -INFINITY;
      m = warp_max(wm);
      s = lane < kWarps && wm > -INFINITY ? s_s[turn][lane] * ex2((wm - m) * kLog2e) : 0.f;
      s = warp_sum(s);
      at = __reduce_min_sync(0xffffffffu, lane < kWarps && wm == m ? s_i[turn][lane] : 0xffffffffu);
      // (the index is not looked at where m is -inf)
      if (lane == 0) a.part[k] = make_float4(m, s, __uint_as_float(static_cast<uint32_t>(b) * a.vocab + v0 + at), 0.f);
    }
  }
}

// A threshold in the candidates' order: a candidate with key words (h, l) and flat
// index f reaches it if it is not behind it.
struct BeamBar {
  uint32_t h, l, f;
  __device__ __forceinline__ bool reached(uint32_t kh, uint32_t kl, uint32_t kf) const {
    return (kh > h) | ((kh == h) & ((kl > l) | ((kl == l) & (kf <= f))));
  }
};

// Sum over the CTA; every thread gets it. red: one word per warp, twice over
// (alternate `turn` between calls, so that one barrier a call is enough).
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t (*red)[kBeamThreads / 32], int turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, red[turn & 1][threadIdx.x & (kBeamThreads / 32 - 1)]) /
         (32 / (kBeamThreads / 32));
}

// Candidates to choose from: n of them in shared memory (a high word of 0 is none;
// the places up to the next multiple of 4 kBeamThreads hold 0), or (LISTS below) the
// lists of all CTAs in the workspace.
struct BeamSource {
  const uint32_t *h, *l, *f;
  int n;
};

// fn(high word, place) of each candidate, and of places without one, whose word is 0;
// places in the lists count through them.
template <bool LISTS, typename Fn>
__device__ __forceinline__ void for_high(const BeamArgs& a, const BeamSource& s, Fn fn) {
  if constexpr (!LISTS) {
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < s.n; i0 += 4 * kBeamThreads) {
      uint32_t k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = s.h[i0 + e * kBeamThreads];
#pragma unroll
      for (int e = 0; e < 4; ++e) fn(k[e], static_cast<size_t>(i0 + e * kBeamThreads));
    }
  } else {
    beam_walk(
        a.slots, a.list, threadIdx.x, [&](int q) { return __ldcg(a.count + q); },
        [&](size_t p) { return __ldcg(a.key + p).x; }, fn);
  }
}

// Scratch of narrow().
struct BeamScratch {
  uint32_t hist[256], red[2][kBeamThreads / 32], found[3];
};

// One more in a bin of the histogram. Lanes that share the first one's bin (equal
// logits) add together.
__device__ __forceinline__ void count_in(uint32_t* hist, uint32_t bin) {
  const uint32_t here = __activemask(), lead = __ffs(here) - 1;
  const bool same = __shfl_sync(here, bin, lead) == bin;
  const uint32_t all = __ballot_sync(here, same);
  if (!same || (threadIdx.x & 31) == lead) atomicAdd(hist + bin, same ? __popc(all) : 1u);
}

// The bar that exactly `want` of the source's (more than want) candidates reach.
// Histograms of 256 bins over ever narrower ranges: of the high words from [lo, hi],
// which holds them all; where equal ones straddle the bar, of their low words,
// then of their inverted indices.
template <bool LISTS>
__device__ __noinline__ BeamBar narrow(const BeamArgs& a, const BeamSource& s, uint32_t want, uint32_t lo, uint32_t hi,
                                       BeamScratch* x) {
  const int tid = threadIdx.x;
  uint32_t above = 0;  // candidates over hi
  uint32_t high = 0, low = 0;
  int level = 0;
#pragma unroll 1
  for (int pass = 0; pass < 12; ++pass) {  // at most four of 8 bits for each word
    const int bits = 32 - __clz(hi - lo), shift = bits > 8 ? bits - 8 : 0;
    __syncthreads();
    if (tid < 256) x->hist[tid] = 0;
    __syncthreads();
    for_high<LISTS>(a, s, [&](uint32_t h, size_t p) {
      uint32_t w = h;
      if (h == 0 || (level > 0 && h != high)) return;
      if (level > 0) {
        w = LISTS ? __ldcg(a.key + p).y : s.l[p];
        if (level > 1) {
          if (w != low) return;
          w = ~(LISTS ? __ldcg(a.flat + p) : s.f[p]);
        }
      }
      if ((w >= lo) & (w <= hi)) count_in(x->hist, (w - lo) >> shift);
    });
    __syncthreads();
    if (tid < 32) {
      // lane l holds bins 8 l .. 8 l + 7; find the bin in which the want-th from above lies
      uint32_t own = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) own += x->hist[8 * tid + j];
      uint32_t over = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_down_sync(0xffffffffu, over, o);
        if (tid + o < 32) over += v;
      }
      over += above - own;  // candidates above this lane's bins
      if (over < want && over + own >= want) {
        int j = 7;
        while (over + x->hist[8 * tid + j] < want) over += x->hist[8 * tid + j--];
        x->found[0] = 8 * tid + j, x->found[1] = over, x->found[2] = x->hist[8 * tid + j];
      }
    }
    __syncthreads();
    lo += x->found[0] << shift;
    above = x->found[1];
    if (above + x->found[2] == want) break;
    if (shift > 0) {
      hi = lo + min(hi - lo, (1u << shift) - 1u);
    } else {  // (indices differ: this ends at level 2 at the latest)
      if (level++ == 0) high = lo; else low = lo;
      lo = 0;
      hi = 0xffffffffu;
      if (level == 2) lo = ~static_cast<uint32_t>(static_cast<uint32_t>(a.beams) * a.vocab - 1u);
    }
  }
  return level == 0 ? BeamBar{lo, 0, 0xffffffffu} : level == 1 ? BeamBar{high, lo, 0xffffffffu} : BeamBar{high, low, ~lo};
}

// Pass 2. Dynamic shared memory: key words and flat indices of the chunks' maxima
// (the words' places hold the maxima and sums first), later of the candidates.
// Short loops rather than unrolled code: what runs once waits for its fetch. The
// registers of a third of an SM: it waits beside kChunkCtas CTAs of pass 1.
__global__ void __launch_bounds__(kBeamThreads, 3) beam_pick_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char beam_raw[];
  uint32_t* sh = reinterpret_cast<uint32_t*>(beam_raw);
  uint32_t *sl = sh + kBeamGather, *sf = sl + kBeamGather;
  float *smax = reinterpret_cast<float*>(sh), *ssum = reinterpret_cast<float*>(sl);
  __shared__ float2 off[kBeamsMax];  // of the rows: score - lse
  __shared__ float rest[kBeamsMax];
  __shared__ BeamScratch scratch;
  __shared__ uint32_t cnt[kBeamThreads / 32], s_lo, s_hi, s_n, s_mine;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kBeamThreads / 32;
  constexpr float kLog2e = 1.44269504088896340736f;
  auto pad = [](int n) { return (n + 4 * kBeamThreads - 1) / (4 * kBeamThreads) * (4 * kBeamThreads); };

  pdl_wait();
  const int padded = pad(a.chunks);
#pragma unroll 1
  for (int k0 = tid; k0 < padded; k0 += 4 * kBeamThreads) {
    float4 p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p[e] = k0 + e * kBeamThreads < a.chunks ? a.part[k0 + e * kBeamThreads] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      smax[k0 + e * kBeamThreads] = p[e].x;
      ssum[k0 + e * kBeamThreads] = p[e].y;
      sf[k0 + e * kBeamThreads] = __float_as_uint(p[e].z);
    }
  }
#pragma unroll 1
  for (int b = tid; b < a.beams; b += kBeamThreads) off[b].x = a.scores[b];
  if (tid == 0) s_mine = s_lo = 0xffffffffu, s_n = s_hi = 0;
  __syncthreads();
  // row offsets, as many lanes a row as there are; -inf where the row offers nothing
  const int lanes = 1 << a.row_lanes;
#pragma unroll 1
  for (int b0 = 0; b0 < a.beams; b0 += kBeamThreads >> a.row_lanes) {
    const int b = b0 + (tid >> a.row_lanes), c0 = (b < a.beams ? b : 0) * a.per_row;
    float m = -INFINITY, s = 0.f;
#pragma unroll 4
    for (int c = tid & (lanes - 1); c < a.per_row; c += lanes) m = fmaxf(m, smax[c0 + c]);
#pragma unroll 1
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m > -INFINITY && m < INFINITY;
#pragma unroll 4
    for (int c = tid & (lanes - 1); c < a.per_row; c += lanes)
      s = fmaf(ssum[c0 + c], ex2((smax[c0 + c] - (finite ? m : 0.f)) * kLog2e), s);
#pragma unroll 1
    for (int o = lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (b < a.beams && (tid & (lanes - 1)) == 0) {
      const float sc = off[b].x;
      float over = 0.f;
      const float2 o = finite && isfinite(sc) ? row_offset(sc, m, s, &over) : make_float2(-INFINITY, 0.f);
      off[b] = isfinite(o.x) ? o : make_float2(-INFINITY, 0.f);
      rest[b] = over;
    }
  }
  __syncthreads();
  // the chunks' keys, and the range of their high words
  uint32_t some = 0, lo = 0xffffffffu, hi = 0;
#pragma unroll 2
  for (int k = tid; k < padded; k += kBeamThreads) {
    const int b = k < a.chunks ? static_cast<int>((k * a.row_inv) >> 32) : 0;
    const float2 o = off[b];
    const float m = smax[k];
    const bool in = (k < a.chunks) & (m > -INFINITY) & (o.x > -INFINITY);
    const uint2 w = key_words(m, o, rest[b]);
    sh[k] = in ? w.x : 0;
    sl[k] = w.y;
    some += in;
    lo = in ? min(lo, w.x) : lo;
    hi = in ? max(hi, w.x) : hi;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    atomicMin(&s_lo, lo);
    atomicMax(&s_hi, hi);
  }
  const uint32_t n_all = block_sum(some, scratch.red, 0);
  // the bar: the n_out-th best of the keys
  BeamBar bar{1, 0, 0xffffffffu};  // reached by every key
  const uint32_t want = a.n_out;
  if (n_all > want) bar = narrow<false>(a, BeamSource{sh, sl, sf, a.chunks}, want, s_lo, s_hi, &scratch);

  // the blockIdx.x-th chunk that reaches the bar, in the order of the chunks: a warp
  // counts those of its range, and the one that holds it finds it
  const int range = padded / kWarps, from = warp * range, until = from + range;
  uint32_t c = 0;
#pragma unroll 4
  for (int k = from + lane; k < until; k += 32) c += (sh[k] != 0) & bar.reached(sh[k], sl[k], sf[k]);
  c = __reduce_add_sync(0xffffffffu, c);
  if (lane == 0) cnt[warp] = c;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? cnt[lane & (kWarps - 1)] : 0);
  if (blockIdx.x >= before && blockIdx.x < before + c) {
    uint32_t at = before;
#pragma unroll 1
    for (int k0 = from; k0 < until; k0 += 32) {
      const int k = k0 + lane;
      const bool in = (sh[k] != 0) & bar.reached(sh[k], sl[k], sf[k]);
      const uint32_t bal = __ballot_sync(0xffffffffu, in);
      if (in && at + __popc(bal & ((1u << lane) - 1u)) == blockIdx.x) s_mine = k;
      at += __popc(bal);
    }
  }
  __syncthreads();
  const uint32_t mine = s_mine, key_lo = bar.h;
  const size_t base = static_cast<size_t>(blockIdx.x) * a.list;
  if (mine != 0xffffffffu) {
    const int b = static_cast<int>((mine * a.row_inv) >> 32), v0 = (mine - b * a.per_row) * a.chunk,
              n = min(a.chunk, a.vocab - v0);
    const float* x = a.logits + a.stride * b + v0;
    const float2 o = off[b];
    const float over = rest[b];
    const uint32_t f0 = static_cast<uint32_t>(b) * a.vocab + v0;
    const float bar_value = bar.h == 1 ? -INFINITY : unorder32(bar.h);
    // y + o.x differs from the key by the offset's remainder and a rounding of each
    const float low = bar_value - (1e-6f * fabsf(bar_value) + 1.001f * fabsf(o.y));
#pragma unroll 1
    for (int i0 = tid * 4; i0 < n; i0 += kBeamThreads * 16) {
      float y[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q * kBeamThreads * 4;
        if (a.vec && i + 4 <= n) {
          const float4 f = *reinterpret_cast<const float4*>(x + i);
          y[4 * q] = f.x, y[4 * q + 1] = f.y, y[4 * q + 2] = f.z, y[4 * q + 3] = f.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[4 * q + e] = i + e < n ? x[i + e] : -INFINITY;
        }
      }
      uint32_t near = 0;  // those that are not masked (a NaN is not) and not clearly below the bar
#pragma unroll
      for (int e = 0; e < 16; ++e)
        near |= static_cast<uint32_t>((y[e] > -INFINITY) & (y[e] + o.x >= low)) << e;
#pragma unroll 1
      for (; near; near &= near - 1) {
        const int e = __ffs(near) - 1, i = i0 + (e >> 2) * kBeamThreads * 4 + (e & 3);
        const uint2 w = key_words(x[i], o, over);
        if (bar.reached(w.x, w.y, f0 + i)) {
          const uint32_t p = atomicAdd(&s_n, 1u);
          a.key[base + p] = w;
          a.flat[base + p] = f0 + i;
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.count[blockIdx.x] = s_n;
    __threadfence();  // after the barrier: the whole CTA's list before its arrival
    s_mine = atomicAdd(a.counter, 1u);
  }
  __syncthreads();
  if (s_mine != gridDim.x - 1) return;
  __threadfence();

  // the last CTA: rank what was listed. Up to kBeamGather candidates are held in
  // shared memory; more of them (many equal logits) are narrowed where they lie.
  uint32_t* first = reinterpret_cast<uint32_t*>(off);  // place of each list's first candidate; later ranks
  uint32_t* taken = first + kBeamOutMax;               // candidates of each rank
  const int q0 = 2 * tid;
  const uint32_t c0 = q0 < a.slots ? __ldcg(a.count + q0) : 0, c1 = q0 + 1 < a.slots ? __ldcg(a.count + q0 + 1) : 0;
  uint32_t sum = c0 + c1;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) cnt[warp] = sum;
  if (tid == 0) s_n = 0;
  taken[tid] = taken[tid + kBeamThreads] = 0;
  __syncthreads();
  const uint32_t part = cnt[lane & (kWarps - 1)];
  const uint32_t listed = __reduce_add_sync(0xffffffffu, lane < kWarps ? part : 0);
  sum += __reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
  first[q0] = sum - c0 - c1, first[q0 + 1] = sum - c1;
  __syncthreads();
  uint32_t n = listed;
  if (listed <= kBeamGather) {
#pragma unroll 1
    for (uint32_t i = tid; i < listed; i += kBeamThreads) {
      int q = 0;  // the list that holds the i-th: the last that begins at or before it
#pragma unroll 1
      for (int step = kBeamOutMax / 2; step > 0; step >>= 1)
        if (q + step < a.slots && first[q + step] <= i) q += step;
      const size_t p = static_cast<size_t>(q) * a.list + (i - first[q]);
      const uint2 w = __ldcg(a.key + p);
      sf[i] = __ldcg(a.flat + p);
      sh[i] = w.x, sl[i] = w.y;
    }
  } else {
    bar = narrow<true>(a, BeamSource{}, want, key_lo, 0xffffffffu, &scratch);
    for_high<true>(a, BeamSource{}, [&](uint32_t h, size_t p) {
      if (h < bar.h) return;  // (0, behind a list's end, is below every bar)
      const uint32_t l = __ldcg(a.key + p).y, f = __ldcg(a.flat + p);
      if (bar.reached(h, l, f)) {
        const uint32_t w = atomicAdd(&s_n, 1u);
        if (w < kBeamGather) sh[w] = h, sl[w] = l, sf[w] = f;
      }
    });
    __syncthreads();
    n = min(s_n, want);
  }
  auto fill = [&]() {  // zeros behind the candidates
#pragma unroll 1
    for (int i = n + tid; i < pad(n); i += kBeamThreads) sh[i] = 0;
    __syncthreads();
  };
  fill();
  if (n > want && n > kBeamRank) {
    // too many to rank against each other: the n_out best, by way of the first lists' places
    bar = narrow<false>(a, BeamSource{sh, sl, sf, static_cast<int>(n)}, want, key_lo, 0xffffffffu, &scratch);
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll 1
    for (uint32_t i = tid; i < n; i += kBeamThreads)
      if (bar.reached(sh[i], sl[i], sf[i])) {
        const uint32_t w = atomicAdd(&s_n, 1u);
        a.key[w] = make_uint2(sh[i], sl[i]);
        a.flat[w] = sf[i];
      }
    __syncthreads();
    n = min(s_n, want);
#pragma unroll 1
    for (uint32_t i = tid; i < n; i += kBeamThreads) sh[i] = a.key[i].x, sl[i] = a.key[i].y, sf[i] = a.flat[i];
    fill();
  }
  // ranks by counting the better ones by their high words, four at a time, `split`
  // threads a candidate; candidates that came to one rank share theirs and compare
  // the rest (n <= kBeamOutMax here)
  int lg = 0;
  while (lg < 5 && (n << (lg + 1)) <= kBeamThreads) ++lg;
  const int split = 1 << lg;
#pragma unroll 1
  for (uint32_t i0 = 0; i0 < n; i0 += kBeamThreads >> lg) {
    const uint32_t i = i0 + (tid >> lg), h = i < n ? sh[i] : 0xffffffffu;
    uint32_t rank = 0;
#pragma unroll 4
    for (uint32_t j = (tid & (split - 1)) * 4; j < n; j += split * 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(sh + j);
      rank += (k.x > h) + (k.y > h) + (k.z > h) + (k.w > h);
    }
#pragma unroll 1
    for (int o = split / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < n && (tid & (split - 1)) == 0) {
      atomicAdd(&taken[rank], 1u);
      first[i] = rank;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (uint32_t i = tid; i < n; i += kBeamThreads) {
    uint32_t rank = first[i];
    if (taken[rank] > 1)
#pragma unroll 4
      for (uint32_t j = 0; j < n; ++j)
        rank += sh[j] == sh[i] && (sl[j] > sl[i] || (sl[j] == sl[i] && sf[j] < sf[i]));
    if (rank < want) {
      a.out_scores[rank] = unorder32(sh[i]);
      a.out_parents[rank] = static_cast<int32_t>(sf[i] / static_cast<uint32_t>(a.vocab));
      a.out_tokens[rank] = static_cast<int32_t>(sf[i] % static_cast<uint32_t>(a.vocab));
    }
  }
#pragma unroll 1
  for (uint32_t i = n + tid; i < want; i += kBeamThreads) {
    a.out_scores[i] = -INFINITY;
    a.out_parents[i] = a.out_tokens[i] = -1;
  }
}

bool select_sizes_ok(const beam_select_args* a) {
  return a->beams >= 1 && a->beams <= kBeamsMax && a->n_out >= 1 && a->n_out <= kBeamOutMax && a->vocab >= 1 &&
         static_cast<long long>(a->beams) * a->vocab < (1ll << 31);
}

// ---- reorder ----------------------------------------------------------------

constexpr int kReorderThreads = 256;

struct ReorderArgs {
  int beams, layers, n_kv;
  int row16;  // 16-byte pieces of one token of one head
  uint4 *k, *v;
  long long layer16;  // pieces between layers
  PagePool pool;
  const int32_t *parents, *spare, *old_table, *old_len;
  int32_t *new_table, *new_len;
  uint32_t* err;
};

// Grid: (beams, layers, 2: keys, values). A tail's tokens are contiguous per
// head: the copy is n_kv runs of rest * row16 16-byte pieces, read and written
// once; bound by memory (64 beams, 28 layers, 24 tokens of 8 heads of 128 in
// bfloat16: 50 us, 7.0 TB/s).
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const ReorderArgs a) {
  const int i = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const bool first = layer == 0 && blockIdx.z == 0;
  pdl_wait();  // the parents and the pages come from the stream's previous kernels
  pdl_trigger();
  const int p = a.parents[i];
  int len = -1, src = -1, dst = -1;
  bool bad = p >= a.beams;
  if (p >= 0 && p < a.beams) len = a.old_len[p];
  const int full = len < 0 ? 0 : len >> a.pool.shift, rest = len < 0 ? 0 : len & ((1 << a.pool.shift) - 1);
  const int32_t* row = a.old_table + static_cast<long long>(p < 0 ? 0 : p) * a.pool.width;
  if (len >= 0) {
    dst = a.spare[i];
    bad = len >= page_capacity(a.pool) || dst < 0 || dst >= a.pool.num_pages;
    if (!bad && rest > 0) {
      src = page_of(a.pool, row, len);
      bad = src < 0;
    }
    const int filled = bad ? 0 : full;
    for (int j = tid; j < filled; j += kReorderThreads) bad |= page_of(a.pool, row, static_cast<int64_t>(j) << a.pool.shift) < 0;
  }
  bad = __syncthreads_or(bad);  // every CTA of the slot comes to the same answer
  if (bad) len = -1;
  if (first) {
    if (bad && tid == 0) atomicOr(a.err, ERR_BAD_PAGE);
    if (tid == 0) a.new_len[i] = len;
    int32_t* out = a.new_table + static_cast<long long>(i) * a.pool.width;
    for (int j = tid; j < a.pool.width; j += kReorderThreads)
      out[j] = len < 0 || j > full ? -1 : j == full ? dst : row[j];
  }
  if (len < 0 || rest == 0) return;
  uint4* pool = (blockIdx.z ? a.v : a.k) + a.layer16 * layer;
  const int run = rest * a.row16;  // pieces per head
  const long long head = static_cast<long long>(a.row16) << a.pool.shift;
  const uint4* s = pool + pool_row(a.pool, src, 0, 0) * a.row16;
  uint4* d = pool + pool_row(a.pool, dst, 0, 0) * a.row16;
  for (int t = tid; t < run * a.n_kv; t += kReorderThreads) {
    const long long at = t / run * head + t % run;
    d[at] = s[at];
  }
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" size_t beam_select_workspace(const beam_select_args* a) {
  if (!a || !select_sizes_ok(a)) return 0;
  return beam_layout(a->beams, a->vocab, a->n_out).total;
}

extern "C" dec_status beam_select(const beam_select_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "beam_select: NULL arguments");
  if (!select_sizes_ok(a))
    return fail(nullptr, DEC_EINVAL, "beam_select: beams %d, vocab %d, n_out %d", a->beams, a->vocab, a->n_out);
  if (!a->logits || !a->scores || !a->out_scores || !a->out_parents || !a->out_tokens)
    return fail(nullptr, DEC_EINVAL, "beam_select: NULL pointer");
  if (a->logits_stride < 0 || (a->beams > 1 && a->logits_stride < a->vocab))
    return fail(nullptr, DEC_EINVAL, "beam_select: rows of %d logits overlap at stride %lld", a->vocab,
                static_cast<long long>(a->logits_stride));
  if (!aligned_to(4, a->logits, a->scores, a->out_scores, a->out_parents, a->out_tokens))
    return fail(nullptr, DEC_EINVAL, "beam_select: a pointer is not aligned to its elements");
  if (!a->d_workspace || reinterpret_cast<uintptr_t>(a->d_workspace) % 256)
    return fail(nullptr, DEC_EINVAL, "beam_select: workspace must be non-NULL and 256-byte aligned");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  const BeamLayout L = beam_layout(a->beams, a->vocab, a->n_out);
  if (a->workspace_bytes < L.total)
    return fail(nullptr, DEC_ENOMEM, "beam_select: workspace has %zu bytes, %zu needed", a->workspace_bytes, L.total);
  char* w = static_cast<char*>(a->d_workspace);
  BeamArgs k{};
  k.beams = a->beams;
  k.vocab = a->vocab;
  k.n_out = a->n_out;
  k.chunk = L.chunk;
  k.per_row = L.per_row;
  k.chunks = L.chunks;
  k.slots = L.slots;
  k.list = L.list;
  k.logits = a->logits;
  k.stride = a->logits_stride;
  k.scores = a->scores;
  k.out_scores = a->out_scores;
  k.out_parents = a->out_parents;
  k.out_tokens = a->out_tokens;
  k.part = reinterpret_cast<float4*>(w + L.part);
  k.counter = reinterpret_cast<uint32_t*>(w + L.counter);
  k.count = reinterpret_cast<uint32_t*>(w + L.count);
  k.key = reinterpret_cast<uint2*>(w + L.key);
  k.flat = reinterpret_cast<uint32_t*>(w + L.flat);
  k.row_inv = (1ull << 32) / L.per_row + 1;
  while (k.row_lanes < 5 && (a->beams << (k.row_lanes + 1)) <= kBeamThreads) ++k.row_lanes;
  k.vec = aligned16(a->logits) && a->logits_stride % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // static and dynamic shared memory together pass the 48 KB that need no opt-in
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    WSG_CUDA_TRY(nullptr, cudaFuncSetAttribute(beam_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBeamSmem));
    // A CTA of pass 2 takes its place beside those of pass 1 only where the SM's
    // shared memory is split for both (without: 15 and 26 us for 4 and 64 beams, with 12 and 23)
    WSG_CUDA_TRY(nullptr, allow_smem_shared(beam_chunks_kernel, 0));
    WSG_CUDA_TRY(nullptr, allow_smem_shared(beam_pick_kernel, 0));
    lifted[di.device] = true;
  }
  const int grid = L.chunks < kChunkCtas * di.sms ? L.chunks : kChunkCtas * di.sms;
  WSG_CUDA_TRY(nullptr, launch_k(beam_chunks_kernel, dim3(grid), dim3(kChunkThreads), 0, s, true, k));
  WSG_CUDA_TRY(nullptr, launch_k(beam_pick_kernel, dim3(L.slots), dim3(kBeamThreads), kBeamSmem, s, true, k));
  return DEC_OK;
}

extern "C" dec_status beam_reorder_pages(const beam_reorder_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: NULL arguments");
  const int shift = page_shift(a->page_size);
  if (a->beams < 0 || a->layers < 1 || a->layers > 65535 || a->n_kv < 1 || a->n_kv > 16384 || a->head_dim < 8 || a->head_dim > 128 ||
      a->head_dim % 8 || (a->kvdtype != DEC_F32 && a->kvdtype != DEC_BF16) || shift < 0 || a->num_pages < 0 ||
      a->table_stride < 1 || a->layer_stride < 0)
    return fail(nullptr, DEC_EINVAL,
                "beam_reorder_pages: beams %d, layers %d, n_kv %d, head_dim %d, kvdtype %d, page_size %d, num_pages %d, "
                "table_stride %d",
                a->beams, a->layers, a->n_kv, a->head_dim, a->kvdtype, a->page_size, a->num_pages, a->table_stride);
  if (a->beams == 0) return DEC_OK;
  if (!a->k_pages || !a->v_pages || !a->parents || !a->spare || !a->old_table || !a->old_len || !a->new_table || !a->new_len)
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: NULL pointer");
  const int elem = a->kvdtype == DEC_F32 ? 4 : 2;
  if (!aligned16(a->k_pages) || !aligned16(a->v_pages) || a->layer_stride * elem % 16)
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: the pools must be 16-byte aligned in every layer");
  if (!aligned_to(4, a->parents, a->spare, a->old_table, a->old_len, a->new_table, a->new_len))
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: a pointer is not aligned to its elements");
  const size_t beams = a->beams, entries = beams * a->table_stride;
  struct Array {
    const int32_t* at;
    size_t n;
  };
  auto overlap = [](Array x, Array y) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(x.at), q = reinterpret_cast<uintptr_t>(y.at);
    return p < q ? q - p < 4 * x.n : p - q < 4 * y.n;
  };
  const Array table{a->new_table, entries}, length{a->new_len, beams};
  if (overlap(table, {a->old_table, entries}) || overlap(length, {a->old_len, beams}))
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: the new table and lengths must not overlap the old");
  const long long layer = static_cast<long long>(a->num_pages) * a->n_kv * a->page_size * a->head_dim;
  if (a->layers > 1 && a->layer_stride < layer)
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: layers of %lld elements overlap at stride %lld", layer,
                static_cast<long long>(a->layer_stride));
  // (a slot's other CTAs may still have to read what its first one writes over)
  for (const Array x : {Array{a->parents, beams}, Array{a->spare, beams}})
    if (overlap(table, x) || overlap(length, x))
      return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: the new table and lengths must not overlap parents or spare pages");
  if (overlap(table, {a->old_len, beams}) || overlap(length, {a->old_table, entries}) || overlap(table, length))
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: tables and lengths must not overlap");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  ReorderArgs k{};
  k.beams = a->beams;
  k.layers = a->layers;
  k.n_kv = a->n_kv;
  k.row16 = a->head_dim * elem / 16;
  k.k = static_cast<uint4*>(a->k_pages);
  k.v = static_cast<uint4*>(a->v_pages);
  k.layer16 = a->layer_stride * elem / 16;
  k.pool = PagePool{a->num_pages, a->n_kv, shift, a->table_stride};
  k.parents = a->parents;
  k.spare = a->spare;
  k.old_table = a->old_table;
  k.old_len = a->old_len;
  k.new_table = a->new_table;
  k.new_len = a->new_len;
  k.err = di.err;
  WSG_CUDA_TRY(nullptr, launch_k(beam_reorder_kernel, dim3(a->beams, a->layers, 2), dim3(kReorderThreads), 0,
                                 static_cast<cudaStream_t>(stream), true, k));
  return DEC_OK;
}
