// beam_select and beam_reorder_pages: beam search's selection over beams and
// vocabulary, and the page tables and tail pages of the beams it leaves.
//
// Selection. A candidate (b, v) has the key score_b + (x_bv - lse_b), lse_b =
// log sum exp x_b. Every logit is read once from memory:
//   pass 1  one CTA per chunk of a row: the chunk's maximum (with its lowest
//           index) and sum of exp(x - maximum), the running pair of a softmax;
//   pass 2  every CTA joins the chunks' pairs into the rows' lse, so that each
//           chunk's maximum becomes a key. The n_out-th best of these keys (by
//           bisection) is a lower bound T of the n_out-th best candidate, and only
//           the at most n_out chunks whose maximum reaches T hold selected ones. CTA i
//           re-reads the i-th of them (from L2) and lists the candidates that
//           reach T; the last CTA to finish narrows the
//           listed ones to n_out in the same way and ranks them.
// Candidates are ordered by (key descending, flat index ascending), a total
// order: T is exact, ties included, and the result does not depend on timing.
#include <cmath>

#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {
namespace {

constexpr int kChunkThreads = 256, kBeamThreads = 512;
constexpr int kBeamPer = 8;                               // chunks a thread of pass 2 holds
constexpr int kBeamChunksMax = kBeamPer * kBeamThreads;  // chunks of one call (all rows)
constexpr int kBeamChunkMin = 1024;
constexpr int kBeamGather = 4096;  // candidates held in shared memory
constexpr int kBeamsMax = 1024, kBeamOutMax = 1024;
// dynamic shared memory of pass 2: the chunks' maxima and sums and the rows' offsets, later the candidates
constexpr size_t kBeamSmem = 12 * kBeamGather;
static_assert(kBeamSmem >= 8 * kBeamChunksMax + 8 * kBeamsMax, "both fit");

// Workspace: chunk maxima, their indices, chunk sums; the arrival counter; per
// qualified chunk a count and a list of (key, flat index).
struct BeamLayout {
  int chunk, per_row, chunks, slots;
  size_t max, idx, sum, counter, count, key, flat, total;
};

BeamLayout beam_layout(int beams, int vocab, int n_out) {
  BeamLayout L{};
  // the smallest power of two within the bound on the number of chunks
  long long c = kBeamChunkMin;
  while (static_cast<long long>(beams) * ((vocab + c - 1) / c) > kBeamChunksMax) c *= 2;
  L.chunk = static_cast<int>(c);
  L.per_row = static_cast<int>((vocab + c - 1) / c);
  L.chunks = L.per_row * beams;
  L.slots = n_out < L.chunks ? n_out : L.chunks;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  L.max = take(sizeof(float) * L.chunks);
  L.idx = take(sizeof(uint32_t) * L.chunks);
  L.sum = take(sizeof(float) * L.chunks);
  L.counter = take(4);
  L.count = take(sizeof(uint32_t) * L.slots);
  const size_t list = static_cast<size_t>(L.slots) * (c < vocab ? c : vocab);
  L.key = take(sizeof(unsigned long long) * list);
  L.flat = take(sizeof(uint32_t) * list);
  L.total = o;
  return L;
}

struct BeamArgs {
  int beams, vocab, n_out, chunk, per_row, chunks, slots, list;
  const float* logits;
  long long stride;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  float *max, *sum;
  uint32_t *idx, *counter, *count, *flat;
  unsigned long long* key;
  int vec;
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

// The key x + off as order bits, off and the sum as two floats (value and
// remainder, 48 bits): the slow double pipe takes 7 times as long here.
__device__ __forceinline__ unsigned long long key_bits(float x, float2 off) {
  const float s = x + off.x, t = s - x;
  const float e = (x - (s - t)) + (off.x - t) + off.y;  // x + off.x - s exactly, then the remainder
  const float hi = s + e, lo = e - (hi - s);
  return static_cast<unsigned long long>(order32(hi)) << 32 | order32(lo);
}

// Pass 1: chunk blockIdx.x of row blockIdx.y, 16 logits a thread at a time. The
// exponentials are 2^((x - m) log2 e) with m the warp's maximum so far.
__global__ void __launch_bounds__(kChunkThreads) beam_chunks_kernel(const BeamArgs a) {
  constexpr int kWarps = kChunkThreads / 32;
  constexpr float kLog2e = 1.44269504088896340736f;
  __shared__ float s_m[kWarps], s_s[kWarps];
  __shared__ uint32_t s_i[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  const int c = blockIdx.x, b = blockIdx.y;
  const int v0 = c * a.chunk, n = min(a.chunk, a.vocab - v0);
  const float* x = a.logits + a.stride * b + v0;
  if (tid == 0 && b == 0 && c == 0) *a.counter = 0;
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
  if (lane == 0) s_m[warp] = m, s_s[warp] = s, s_i[warp] = at;
  __syncthreads();
  if (warp == 0) {
    const float wm = lane < kWarps ? s_m[lane] : -INFINITY;
    m = warp_max(wm);
    s = lane < kWarps && wm > -INFINITY ? s_s[lane] * ex2((wm - m) * kLog2e) : 0.f;
    s = warp_sum(s);
    at = __reduce_min_sync(0xffffffffu, lane < kWarps && wm == m ? s_i[lane] : 0xffffffffu);
    if (lane == 0) {
      const int k = b * a.per_row + c;
      a.max[k] = m;
      a.sum[k] = s;
      a.idx[k] = static_cast<uint32_t>(b) * a.vocab + v0 + at;  // not looked at where m is -inf
    }
  }
}

// Whether candidate (k, f) is at least (key, index) in the candidates' order.
__device__ __forceinline__ bool reaches(unsigned long long k, uint32_t f, unsigned long long key, uint32_t index) {
  return k > key || (k == key && f <= index);
}

// Sum over the CTA; every thread gets it. red: one word per warp, twice over
// (alternate `turn` between calls, so that one barrier a call is enough).
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t (*red)[kBeamThreads / 32], int turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, red[turn & 1][threadIdx.x & (kBeamThreads / 32 - 1)]) /
         (32 / (kBeamThreads / 32));
}

// Smallest and largest of the CTA's values (lo: ~0 and hi: 0 where a thread has
// none); red64: two words per warp.
__device__ __forceinline__ void block_range(unsigned long long* lo, unsigned long long* hi, unsigned long long* red64) {
  constexpr int kWarps = kBeamThreads / 32;
  unsigned long long l = *lo, h = *hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long l2 = __shfl_xor_sync(0xffffffffu, l, o), h2 = __shfl_xor_sync(0xffffffffu, h, o);
    l = l2 < l ? l2 : l;
    h = h2 > h ? h2 : h;
  }
  if ((threadIdx.x & 31) == 0) red64[threadIdx.x >> 5] = l, red64[kWarps + (threadIdx.x >> 5)] = h;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    l = red64[w] < l ? red64[w] : l;
    h = red64[kWarps + w] > h ? red64[kWarps + w] : h;
  }
  __syncthreads();
  *lo = l;
  *hi = h;
}

// The composite (key, index) that exactly `want` of the CTA's n_all > want
// entries reach: bisection over the keys, from their range [lo, hi], until that
// many reach a key; where equal keys straddle it, over their indices.
// reach(key): how many of this thread's entries have at least this key;
// equal(key, index): how many have this key and at most this index.
template <typename Reach, typename Equal>
__device__ __forceinline__ void bisect(uint32_t want, uint32_t n_all, unsigned long long lo, unsigned long long hi,
                                       Reach reach, Equal equal, uint32_t (*red)[kBeamThreads / 32], int* turn,
                                       unsigned long long* key, uint32_t* index) {
  unsigned long long end = hi + 1;  // n(lo) >= want > n(end)
  uint32_t n_lo = n_all, n_end = 0;
  while (n_lo != want && end - lo > 1) {
    const unsigned long long mid = lo + (end - lo) / 2;
    const uint32_t n = block_sum(reach(mid), red, (*turn)++);
    if (n >= want)
      lo = mid, n_lo = n;
    else
      end = mid, n_end = n;
  }
  *key = lo;
  *index = 0xffffffffu;
  if (n_lo == want) return;
  uint32_t i0 = 0, i1 = 0xffffffffu;  // the want - n_end lowest indices with key lo
  while (i0 < i1) {
    const uint32_t mid = i0 + (i1 - i0) / 2;
    if (block_sum(equal(lo, mid), red, (*turn)++) >= want - n_end)
      i1 = mid;
    else
      i0 = mid + 1;
  }
  *index = i1;
}

// Pass 2. Dynamic shared memory: offsets of the rows, maxima and sums of the
// chunks.
__global__ void __launch_bounds__(kBeamThreads) beam_pick_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char beam_raw[];
  float2* off = reinterpret_cast<float2*>(beam_raw);  // of the rows: score - lse
  float* cmax = reinterpret_cast<float*>(off + a.beams);
  float* csum = cmax + a.chunks;
  // the last CTA's candidates, in the place of the chunks' maxima and sums
  unsigned long long* gkey = reinterpret_cast<unsigned long long*>(beam_raw);
  uint32_t* gidx = reinterpret_cast<uint32_t*>(gkey + kBeamGather);
  __shared__ unsigned long long red64[2 * kBeamThreads / 32];
  __shared__ uint32_t red[2][kBeamThreads / 32], cnt[kBeamPer * kBeamThreads / 32];
  __shared__ uint32_t s_n, s_mine;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kBeamThreads / 32;

  pdl_wait();
  uint32_t cidx[kBeamPer];  // this thread's chunks: tid, tid + kBeamThreads, ...
#pragma unroll
  for (int j = 0; j < kBeamPer; ++j) {
    const int k = tid + j * kBeamThreads;
    cidx[j] = 0;
    if (k < a.chunks) {
      cmax[k] = a.max[k];
      csum[k] = a.sum[k];
      cidx[j] = a.idx[k];
    }
  }
  if (tid == 0) s_mine = 0xffffffffu, s_n = 0;
  __syncthreads();
  // row offsets score - lse; -inf where the row offers nothing
  for (int b = warp; b < a.beams; b += kWarps) {
    const float* rm = cmax + b * a.per_row;
    float m = -INFINITY;
    for (int c = lane; c < a.per_row; c += 32) m = fmaxf(m, rm[c]);
    m = warp_max(m);
    float s = 0.f;
    if (m > -INFINITY && m < INFINITY)
      for (int c = lane; c < a.per_row; c += 32) s += csum[b * a.per_row + c] * expf(rm[c] - m);
    s = warp_sum(s);
    if (lane == 0) off[b] = make_float2(m, s);
  }
  __syncthreads();
  for (int b = tid; b < a.beams; b += kBeamThreads) {
    // score - (m + log s), s = 2^e f with f in [0.7, 1.42): log f is below 0.36, so a
    // float32 logarithm of it is good to 3e-8
    const float m = off[b].x, s = off[b].y, sc = a.scores[b];
    float2 o = make_float2(-INFINITY, 0.f);
    if (m > -INFINITY && m < INFINITY && isfinite(sc)) {
      int e;
      float f = frexpf(s, &e);
      if (f < 0.70710678f) f *= 2.f, --e;
      const double d = static_cast<double>(sc) - (static_cast<double>(m) + e * 0.69314718055994530942 + logf(f));
      o.x = static_cast<float>(d);
      o.y = static_cast<float>(d - static_cast<double>(o.x));
    }
    off[b] = o;
  }
  __syncthreads();
  unsigned long long key[kBeamPer];  // of the chunks' maxima, 0: offers nothing
  unsigned long long lo = ~0ull, hi = 0;
#pragma unroll
  for (int j = 0; j < kBeamPer; ++j) {
    const int k = tid + j * kBeamThreads;
    key[j] = 0;
    if (k < a.chunks) {
      const float2 o = off[k / a.per_row];
      if (cmax[k] > -INFINITY && o.x > -INFINITY) key[j] = key_bits(cmax[k], o);
    }
    if (key[j]) {
      lo = key[j] < lo ? key[j] : lo;
      hi = key[j] > hi ? key[j] : hi;
    }
  }
  // threshold: the n_out-th best of the keys
  uint32_t n_all = 0;
#pragma unroll
  for (int j = 0; j < kBeamPer; ++j) n_all += key[j] != 0;
  int turn = 0;
  n_all = block_sum(n_all, red, turn++);
  unsigned long long tk = 1;  // reached by every key
  uint32_t ti = 0xffffffffu;
  const uint32_t want = a.n_out;
  if (n_all > want) {
    block_range(&lo, &hi, red64);
    bisect(
        want, n_all, lo, hi,
        [&](unsigned long long mid) {
          uint32_t n = 0;
#pragma unroll
          for (int j = 0; j < kBeamPer; ++j) n += key[j] >= mid;
          return n;
        },
        [&](unsigned long long k, uint32_t mid) {
          uint32_t n = 0;
#pragma unroll
          for (int j = 0; j < kBeamPer; ++j) n += key[j] == k && cidx[j] <= mid;
          return n;
        },
        red, &turn, &tk, &ti);
  }

  // the blockIdx.x-th chunk whose maximum reaches the threshold, counted in the
  // order (j, thread); all CTAs count alike
  uint32_t bal[kBeamPer];
#pragma unroll
  for (int j = 0; j < kBeamPer; ++j) {
    bal[j] = __ballot_sync(0xffffffffu, key[j] != 0 && reaches(key[j], cidx[j], tk, ti));
    if (lane == 0) cnt[j * kWarps + warp] = __popc(bal[j]);
  }
  __syncthreads();
  {
    uint32_t before = 0;
#pragma unroll
    for (int j = 0; j < kBeamPer; ++j) {
      const uint32_t c = lane < kWarps ? cnt[j * kWarps + lane] : 0;
      const uint32_t mine = before + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
      before += __reduce_add_sync(0xffffffffu, c);
      if (((bal[j] >> lane) & 1u) && mine + __popc(bal[j] & ((1u << lane) - 1u)) == blockIdx.x)
        s_mine = tid + j * kBeamThreads;
    }
  }
  __syncthreads();
  const uint32_t mine = s_mine;
  const size_t base = static_cast<size_t>(blockIdx.x) * a.list;
  if (mine != 0xffffffffu) {
    const int b = mine / a.per_row, v0 = (mine % a.per_row) * a.chunk, n = min(a.chunk, a.vocab - v0);
    const float* x = a.logits + a.stride * b + v0;
    const float2 o = off[b];
    const uint32_t f0 = static_cast<uint32_t>(b) * a.vocab + v0;
    for (int i0 = tid; i0 < n; i0 += kBeamThreads * 8) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = i0 + e * kBeamThreads < n ? masked(x[i0 + e * kBeamThreads]) : -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t f = f0 + i0 + e * kBeamThreads;
        const unsigned long long k = key_bits(y[e], o);
        if (y[e] > -INFINITY && reaches(k, f, tk, ti)) {
          const uint32_t p = atomicAdd(&s_n, 1u);
          a.key[base + p] = k;
          a.flat[base + p] = f;
        }
      }
    }
  }
  __threadfence();  // each thread's listed candidates, before the CTA's arrival
  __syncthreads();
  if (tid == 0) {
    a.count[blockIdx.x] = s_n;
    __threadfence();
    s_mine = atomicAdd(a.counter, 1u);
  }
  __syncthreads();
  if (s_mine != gridDim.x - 1) return;
  __threadfence();

  // the last CTA: narrow what was listed to the n_out best and rank them. Up to
  // kBeamGather candidates are held in shared memory; of more (many equal
  // logits) the lists are bisected where they lie.
  if (tid == 0) s_n = 0;
  uint32_t listed = 0;
  for (int q = tid; q < a.slots; q += kBeamThreads) listed += __ldcg(a.count + q);
  listed = block_sum(listed, red, turn++);
  unsigned long long lk = 1;
  uint32_t li = 0xffffffffu;
  // four threads a list: fn(key bits, flat index) of each listed candidate
  auto each = [&](auto fn) {
    for (int q = tid >> 2; q < a.slots; q += kBeamThreads / 4) {
      const uint32_t n = __ldcg(a.count + q);
      for (uint32_t i = tid & 3; i < n; i += 4) {
        const size_t p = static_cast<size_t>(q) * a.list + i;
        fn(__ldcg(a.key + p), __ldcg(a.flat + p));
      }
    }
  };
  if (listed > kBeamGather) {
    lo = ~0ull, hi = 0;
    each([&](unsigned long long k, uint32_t) { lo = k < lo ? k : lo, hi = k > hi ? k : hi; });
    block_range(&lo, &hi, red64);
    bisect(
        want, listed, lo, hi,
        [&](unsigned long long mid) {
          uint32_t n = 0;
          each([&](unsigned long long k, uint32_t) { n += k >= mid; });
          return n;
        },
        [&](unsigned long long at, uint32_t mid) {
          uint32_t n = 0;
          each([&](unsigned long long k, uint32_t f) { n += k == at && f <= mid; });
          return n;
        },
        red, &turn, &lk, &li);
  }
  each([&](unsigned long long k, uint32_t f) {
    if (reaches(k, f, lk, li)) {
      const uint32_t w = atomicAdd(&s_n, 1u);
      gkey[w] = k;
      gidx[w] = f;
    }
  });
  __syncthreads();
  uint32_t n = s_n;
  if (n > want) {
    unsigned long long k[kBeamGather / kBeamThreads];
    lo = ~0ull, hi = 0;
#pragma unroll
    for (int j = 0; j < kBeamGather / kBeamThreads; ++j) {
      const uint32_t i = tid + j * kBeamThreads;
      k[j] = i < n ? gkey[i] : 0;
      if (k[j]) lo = k[j] < lo ? k[j] : lo, hi = k[j] > hi ? k[j] : hi;
    }
    block_range(&lo, &hi, red64);
    bisect(
        want, n, lo, hi,
        [&](unsigned long long mid) {
          uint32_t c = 0;
#pragma unroll
          for (int j = 0; j < kBeamGather / kBeamThreads; ++j) c += k[j] >= mid;
          return c;
        },
        [&](unsigned long long at, uint32_t mid) {
          uint32_t c = 0;
#pragma unroll
          for (int j = 0; j < kBeamGather / kBeamThreads; ++j) c += k[j] == at && gidx[tid + j * kBeamThreads] <= mid;
          return c;
        },
        red, &turn, &lk, &li);
    // the survivors, in place of the candidates
    uint32_t f[kBeamGather / kBeamThreads];
#pragma unroll
    for (int j = 0; j < kBeamGather / kBeamThreads; ++j) {
      const uint32_t i = tid + j * kBeamThreads;
      f[j] = i < n ? gidx[i] : 0;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBeamGather / kBeamThreads; ++j)
      if (k[j] && reaches(k[j], f[j], lk, li)) {
        const uint32_t w = atomicAdd(&s_n, 1u);
        gkey[w] = k[j];
        gidx[w] = f[j];
      }
    __syncthreads();
    n = s_n;
  }
  // ranks by counting, `split` threads a candidate
  int split = 1;
  while (split < 32 && n * split * 2 <= kBeamThreads) split *= 2;
  for (uint32_t i0 = 0; i0 < n; i0 += kBeamThreads / split) {
    const uint32_t i = i0 + tid / split;
    int rank = 0;
    if (i < n)
      for (uint32_t j = tid % split; j < n; j += split)
        rank += gkey[j] > gkey[i] || (gkey[j] == gkey[i] && gidx[j] < gidx[i]);
    for (int o = split / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < n && tid % split == 0) {
      a.out_scores[rank] = unorder32(static_cast<uint32_t>(gkey[i] >> 32));
      a.out_parents[rank] = static_cast<int32_t>(gidx[i] / static_cast<uint32_t>(a.vocab));
      a.out_tokens[rank] = static_cast<int32_t>(gidx[i] % static_cast<uint32_t>(a.vocab));
    }
  }
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
// once; bound by memory.
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const ReorderArgs a) {
  const int i = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const bool first = layer == 0 && blockIdx.z == 0;
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
  }
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
  k.list = L.chunk < a->vocab ? L.chunk : a->vocab;
  k.logits = a->logits;
  k.stride = a->logits_stride;
  k.scores = a->scores;
  k.out_scores = a->out_scores;
  k.out_parents = a->out_parents;
  k.out_tokens = a->out_tokens;
  k.max = reinterpret_cast<float*>(w + L.max);
  k.idx = reinterpret_cast<uint32_t*>(w + L.idx);
  k.sum = reinterpret_cast<float*>(w + L.sum);
  k.counter = reinterpret_cast<uint32_t*>(w + L.counter);
  k.count = reinterpret_cast<uint32_t*>(w + L.count);
  k.key = reinterpret_cast<unsigned long long*>(w + L.key);
  k.flat = reinterpret_cast<uint32_t*>(w + L.flat);
  k.vec = aligned16(a->logits) && a->logits_stride % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // static and dynamic shared memory together pass the 48 KB that need no opt-in
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    WSG_CUDA_TRY(nullptr, cudaFuncSetAttribute(beam_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBeamSmem));
    lifted[di.device] = true;
  }
  WSG_CUDA_TRY(nullptr, launch_k(beam_chunks_kernel, dim3(L.per_row, a->beams), dim3(kChunkThreads), 0, s, false, k));
  WSG_CUDA_TRY(nullptr, launch_k(beam_pick_kernel, dim3(L.slots), dim3(kBeamThreads), kBeamSmem, s, true, k));
  return DEC_OK;
}

extern "C" dec_status beam_reorder_pages(const beam_reorder_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: NULL arguments");
  const int shift = page_shift(a->page_size);
  if (a->beams < 0 || a->layers < 1 || a->layers > 65535 || a->n_kv < 1 || a->head_dim < 8 || a->head_dim > 128 ||
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
  if (a->new_table == a->old_table || a->new_len == a->old_len)
    return fail(nullptr, DEC_EINVAL, "beam_reorder_pages: the new table and lengths must be other buffers than the old");
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
                                 static_cast<cudaStream_t>(stream), false, k));
  return DEC_OK;
}
