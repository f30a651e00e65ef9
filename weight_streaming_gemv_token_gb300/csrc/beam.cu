// beam_select and beam_reorder_pages: beam search's selection over beams and
// vocabulary, and the page tables and tail pages of the beams it leaves.
//
// Selection. A candidate (b, v) has the key score_b + (x_bv - lse_b), lse_b =
// log sum exp x_b. Every logit is read once from memory:
//   pass 1  one CTA per chunk of a row: the chunk's maximum (with its lowest
//           index) and sum of exp(x - maximum), the running pair of a softmax;
//   pass 2  every CTA joins the chunks' pairs into the rows' lse, so that each
//           chunk's maximum becomes a key. The n_out-th best of these keys is a
//           lower bound T of the n_out-th best candidate, and only the at most
//           n_out chunks whose maximum reaches T can hold a selected one. CTA i
//           re-reads the i-th of them (from L2) and lists the candidates that
//           reach T; the last CTA to finish ranks the listed ones.
// Keys are doubles over (key descending, flat index ascending), a total order:
// T is exact, ties included, and the result does not depend on timing. Usually
// little more than n_out candidates are listed (random logits); equal logits
// can list whole chunks, which the last CTA then narrows digit by digit.
#include <cmath>

#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {
namespace {

constexpr int kBeamThreads = 512;
constexpr int kBeamChunksMax = 4096;  // chunks of one call (all rows)
constexpr int kBeamChunkMin = 1024;
constexpr int kBeamRankMax = 2048;  // candidates ranked directly
constexpr int kBeamsMax = 1024, kBeamOutMax = 1024;
constexpr size_t kBeamSmemMax = 12 * kBeamChunksMax + 8 * kBeamsMax;  // dynamic shared memory of pass 2

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
  L.key = take(sizeof(double) * list);
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
  double* key;
  int vec;
};

// Masked logits (NaN as well) count as -inf.
__device__ __forceinline__ float masked(float x) { return x == x ? x : -INFINITY; }

// A double as an integer in the same order; never 0 for a number.
__device__ __forceinline__ unsigned long long order_bits(double d) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(d));
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// Pass 1: chunk blockIdx.x of row blockIdx.y.
__global__ void __launch_bounds__(kBeamThreads) beam_chunks_kernel(const BeamArgs a) {
  __shared__ float s_m[kBeamThreads / 32], s_s[kBeamThreads / 32];
  __shared__ uint32_t s_i[kBeamThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, b = blockIdx.y;
  const int v0 = c * a.chunk, n = min(a.chunk, a.vocab - v0);
  const float* x = a.logits + a.stride * b + v0;
  if (tid == 0 && b == 0 && c == 0) *a.counter = 0;
  float m = -INFINITY, s = 0.f;
  uint32_t at = 0;
  auto take = [&](float y, int i) {
    y = masked(y);
    if (y > m) {
      s = s * expf(m - y) + 1.f;
      m = y;
      at = i;
    } else if (y > -INFINITY) {
      s += expf(y - m);
    }
  };
  if (a.vec) {
    for (int i = tid * 4; i < n; i += kBeamThreads * 4) {
      if (i + 4 <= n) {
        const float4 y = *reinterpret_cast<const float4*>(x + i);
        take(y.x, i), take(y.y, i + 1), take(y.z, i + 2), take(y.w, i + 3);
      } else {
        for (int j = i; j < n; ++j) take(x[j], j);
      }
    }
  } else {
    for (int i = tid; i < n; i += kBeamThreads) take(x[i], i);
  }
  // joins two (maximum, lowest index, sum) triples; a maximum of -inf has sum 0
  auto join = [&](float m2, uint32_t i2, float s2) {
    if (m2 > m) {
      s = s * expf(m - m2) + s2;
      m = m2;
      at = i2;
    } else {
      if (m2 > -INFINITY) s += s2 * expf(m2 - m);
      if (m2 == m && i2 < at) at = i2;
    }
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const uint32_t i2 = __shfl_xor_sync(0xffffffffu, at, o);
    join(m2, i2, s2);
  }
  if (lane == 0) s_m[warp] = m, s_s[warp] = s, s_i[warp] = at;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kBeamThreads / 32; ++w) join(s_m[w], s_i[w], s_s[w]);
    const int k = b * a.per_row + c;
    a.max[k] = m;
    a.sum[k] = s;
    a.idx[k] = static_cast<uint32_t>(b) * a.vocab + v0 + at;
  }
}

// The composite (key, flat index) of the n-th best of count entries (n >= 1) in
// (key descending, index ascending) order; get(i, &key, &index) gives entry i,
// key 0 for none. Digit by digit from the top over 64 bits of the key, then 32 of
// the inverted index. Entries that reach the result are (key, index) >= it in
// that order. With fewer than n entries: (1, 0xffffffff), which all entries reach.
template <typename Get>
__device__ void nth_best(int n, int count, Get get, uint32_t* hist, unsigned long long* share, unsigned long long* key,
                         uint32_t* index) {
  const int tid = threadIdx.x;
  unsigned long long want_k = 0;  // digits found so far
  uint32_t want_i = 0;            // of ~index
  int left = n;
  for (int digit = 0; digit < 12; ++digit) {
    for (int i = tid; i < 256; i += kBeamThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += kBeamThreads) {
      unsigned long long k;
      uint32_t f;
      get(i, &k, &f);
      if (k == 0) continue;
      bool in;
      uint32_t d;
      if (digit < 8) {
        in = digit == 0 || (k >> (64 - 8 * digit)) == (want_k >> (64 - 8 * digit));
        d = static_cast<uint32_t>(k >> (56 - 8 * digit)) & 255u;
      } else {
        const int e = digit - 8;
        in = k == want_k && (e == 0 || (~f >> (32 - 8 * e)) == (want_i >> (32 - 8 * e)));
        d = (~f >> (24 - 8 * e)) & 255u;
      }
      if (in) atomicAdd(&hist[d], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // suffix sums: lane l holds digits 8 l .. 8 l + 7
      uint32_t own = 0;
      for (int j = 0; j < 8; ++j) own += hist[8 * tid + j];
      uint32_t above = own;  // becomes the count in lanes >= tid
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_down_sync(0xffffffffu, above, o);
        if (tid + o < 32) above += t;
      }
      const uint32_t total = __shfl_sync(0xffffffffu, above, 0);
      if (tid == 0 && total < static_cast<uint32_t>(left)) share[0] = 512;  // all of them
      above -= own;
      for (int j = 7; j >= 0; --j) {
        const uint32_t h = hist[8 * tid + j];
        if (above < static_cast<uint32_t>(left) && above + h >= static_cast<uint32_t>(left))
          share[0] = 8 * tid + j + (above + h == static_cast<uint32_t>(left) ? 256 : 0), share[1] = above;
        above += h;
      }
    }
    __syncthreads();
    const uint32_t r = static_cast<uint32_t>(share[0]);
    const int skipped = static_cast<int>(share[1]);
    __syncthreads();
    if (r == 512) {
      *key = 1, *index = 0xffffffffu;
      return;
    }
    left -= skipped;
    if (digit < 8)
      want_k |= static_cast<unsigned long long>(r & 255u) << (56 - 8 * digit);
    else
      want_i |= (r & 255u) << (24 - 8 * (digit - 8));
    if (r & 256u) break;  // every entry with these digits is among the n best
  }
  *key = want_k;
  *index = ~want_i;
}

// Whether (k, f) is at least (key, index) in the order of nth_best.
__device__ __forceinline__ bool reaches(unsigned long long k, uint32_t f, unsigned long long key, uint32_t index) {
  return k > key || (k == key && f <= index);
}

// Pass 2. Dynamic shared memory: offsets of the rows (double), keys and indices
// of the chunk maxima.
__global__ void __launch_bounds__(kBeamThreads) beam_pick_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char beam_raw[];
  double* off = reinterpret_cast<double*>(beam_raw);
  unsigned long long* ckey = reinterpret_cast<unsigned long long*>(off + a.beams);
  uint32_t* cidx = reinterpret_cast<uint32_t*>(ckey + a.chunks);
  __shared__ unsigned long long rkey[kBeamRankMax];
  __shared__ uint32_t ridx[kBeamRankMax];
  __shared__ uint32_t hist[256];
  __shared__ unsigned long long share[2];
  __shared__ uint32_t s_n, s_mine;
  __shared__ int s_warp[kBeamThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_wait();
  // row offsets score - lse; -inf where the row offers nothing
  for (int b = warp; b < a.beams; b += kBeamThreads / 32) {
    float m = -INFINITY;
    for (int c = lane; c < a.per_row; c += 32) m = fmaxf(m, a.max[b * a.per_row + c]);
    m = warp_max(m);
    float s = 0.f;
    if (m > -INFINITY && m < INFINITY)
      for (int c = lane; c < a.per_row; c += 32) s += a.sum[b * a.per_row + c] * expf(a.max[b * a.per_row + c] - m);
    s = warp_sum(s);
    if (lane == 0) {
      const float sc = a.scores[b];
      const bool ok = m > -INFINITY && m < INFINITY && isfinite(sc);
      off[b] = ok ? static_cast<double>(sc) - (static_cast<double>(m) + log(static_cast<double>(s))) : -INFINITY;
    }
  }
  __syncthreads();
  for (int k = tid; k < a.chunks; k += kBeamThreads) {
    const float m = a.max[k];
    const double o = off[k / a.per_row];
    ckey[k] = m > -INFINITY && o > -INFINITY ? order_bits(static_cast<double>(m) + o) : 0;
    cidx[k] = a.idx[k];
  }
  __syncthreads();
  unsigned long long tk;
  uint32_t ti;
  nth_best(a.n_out, a.chunks, [&](int i, unsigned long long* k, uint32_t* f) { *k = ckey[i], *f = cidx[i]; }, hist, share,
           &tk, &ti);

  // the blockIdx.x-th chunk whose maximum reaches the threshold
  if (tid == 0) s_mine = 0xffffffffu, s_n = 0;
  __syncthreads();
  int before = 0;
  for (int k0 = 0; k0 < a.chunks; k0 += kBeamThreads) {
    const int k = k0 + tid;
    const bool in = k < a.chunks && ckey[k] != 0 && reaches(ckey[k], cidx[k], tk, ti);
    const uint32_t bal = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp] = __popc(bal);
    __syncthreads();
    int at = before, all = 0;
    for (int w = 0; w < kBeamThreads / 32; ++w) {
      if (w < warp) at += s_warp[w];
      all += s_warp[w];
    }
    if (in && at + __popc(bal & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.x)) s_mine = k;
    before += all;
    __syncthreads();
  }
  const uint32_t mine = s_mine;
  const size_t base = static_cast<size_t>(blockIdx.x) * a.list;
  if (mine != 0xffffffffu) {
    const int b = mine / a.per_row, v0 = (mine % a.per_row) * a.chunk, n = min(a.chunk, a.vocab - v0);
    const float* x = a.logits + a.stride * b + v0;
    const double o = off[b];
    for (int i = tid; i < n; i += kBeamThreads) {
      const float y = masked(x[i]);
      const uint32_t f = static_cast<uint32_t>(b) * a.vocab + v0 + i;
      const unsigned long long k = order_bits(static_cast<double>(y) + o);
      if (y > -INFINITY && reaches(k, f, tk, ti)) {
        const uint32_t p = atomicAdd(&s_n, 1u);
        a.key[base + p] = static_cast<double>(y) + o;
        a.flat[base + p] = f;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.count[blockIdx.x] = s_n;
    __threadfence();
    s_mine = atomicAdd(a.counter, 1u);
  }
  __syncthreads();
  if (s_mine != gridDim.x - 1) return;
  __threadfence();

  // the last CTA: rank what was listed
  if (tid == 0) s_n = 0;
  __syncthreads();
  uint32_t total = 0;
  for (int q = 0; q < a.slots; ++q) total += __ldcg(a.count + q);
  unsigned long long lk = 1;
  uint32_t li = 0xffffffffu;
  if (total > kBeamRankMax)
    nth_best(a.n_out, a.slots * a.list,
             [&](int i, unsigned long long* k, uint32_t* f) {
               const int q = i / a.list;
               const bool in = static_cast<uint32_t>(i - q * a.list) < __ldcg(a.count + q);
               *k = in ? order_bits(__ldcg(a.key + i)) : 0;
               *f = in ? __ldcg(a.flat + i) : 0;
             },
             hist, share, &lk, &li);
  for (int q = warp; q < a.slots; q += kBeamThreads / 32) {
    const uint32_t n = __ldcg(a.count + q);
    for (uint32_t i = lane; i < n; i += 32) {
      const size_t p = static_cast<size_t>(q) * a.list + i;
      const unsigned long long k = order_bits(__ldcg(a.key + p));
      const uint32_t f = __ldcg(a.flat + p);
      if (reaches(k, f, lk, li)) {
        const uint32_t w = atomicAdd(&s_n, 1u);
        rkey[w] = k;
        ridx[w] = f;
      }
    }
  }
  __syncthreads();
  const int n = static_cast<int>(s_n);
  for (int i = tid; i < n; i += kBeamThreads) {
    const unsigned long long k = rkey[i];
    const uint32_t f = ridx[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += rkey[j] > k || (rkey[j] == k && ridx[j] < f);
    if (rank < a.n_out) {
      const unsigned long long u = k >> 63 ? k & 0x7fffffffffffffffull : ~k;
      a.out_scores[rank] = static_cast<float>(__longlong_as_double(static_cast<long long>(u)));
      a.out_parents[rank] = static_cast<int32_t>(f / static_cast<uint32_t>(a.vocab));
      a.out_tokens[rank] = static_cast<int32_t>(f % static_cast<uint32_t>(a.vocab));
    }
  }
  for (int i = n + tid; i < a.n_out; i += kBeamThreads) {
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
  k.key = reinterpret_cast<double*>(w + L.key);
  k.flat = reinterpret_cast<uint32_t*>(w + L.flat);
  k.vec = aligned16(a->logits) && a->logits_stride % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = sizeof(double) * L.chunks + sizeof(uint32_t) * L.chunks + sizeof(double) * a->beams;
  // static and dynamic shared memory together pass the 48 KB that need no opt-in
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    WSG_CUDA_TRY(nullptr, allow_smem(beam_pick_kernel, kBeamSmemMax));
    lifted[di.device] = true;
  }
  WSG_CUDA_TRY(nullptr, launch_k(beam_chunks_kernel, dim3(L.per_row, a->beams), dim3(kBeamThreads), 0, s, false, k));
  WSG_CUDA_TRY(nullptr, launch_k(beam_pick_kernel, dim3(L.slots), dim3(kBeamThreads), smem, s, true, k));
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
