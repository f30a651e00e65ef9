// logits_adjust: penalties for repeated tokens, biases and masks of allowed tokens
// on the logits, and the greedy token of what results ("Megakernels", "GPU-wide
// end-to-end generation": greedy argmax on the GPU, lowest ID on ties).
//
// Mathematics, for token v of a row: x = x / rep or x * rep (v in the text), x - freq
// n(v), x - pres (n(v) > 0), x + bias, -inf (not allowed), each step rounded to
// float32 as the definition says.
//
// A cluster of CTAs takes a group of consecutive rows; its CTAs take spans of 512 tokens
// in turn (frequent tokens have neighbouring numbers: with a range each, the first CTA
// had most of a text's). For its tokens a CTA keeps one word each in shared memory: the
// times that the token came (bits 0-19), the number of its bias in the list (20-29) and
// whether the prompt has it (31; 30: its drafted part), built once a request from its text, by
// integer atomics whose order does not matter, and a list of those that have one. A row then is
//   - a copy of all tokens without a rule but the mask, four a thread;
//   - the listed tokens, one a thread, so that the long division runs in full warps;
//   - the tokens drafted on the way to the row, which are listed apart for every row.
// They touch different tokens, so rows need no barrier between them and a CTA's warps drift
// apart over their loads. The logits are read and written once and nothing is kept between
// calls. The CTAs' best tokens, as (order-preserving bits of the value, inverted token), meet
// in the first CTA's shared memory.
//
// Bound by memory for many rows, by a chain of latencies (text, logits, cluster) for one.
// Measured, 177 rows of 32 requests with 3,000 tokens of text each: 62 us (3.5 TB/s, 44% of the
// issue slots, a quarter of the warps' time at the barriers of a request's words); every token's
// rules in the copy 78; with a range of the vocabulary a CTA and no barriers 105.
#include "common.h"
#include "ptx.cuh"
#include "spans.h"

namespace wsg {
namespace {

constexpr int kLaThreads = 512, kLaWarps = kLaThreads / 32, kLaCluster = 8, kLaChunkMax = 20480, kLaRows = 8;
constexpr int kLaBatch = 5;      // quads of logits a thread asks for at a time
constexpr int kLaSpan = 9;        // log2 of the tokens of a span
constexpr int kLaDrafts = 256;   // drafted tokens of a row of a CTA's that are listed
constexpr int kLaTouched = 2048; // tokens with a word that are listed
constexpr int kLaTextMax = 1 << 19, kLaDraftMax = (1 << 19) - 1, kLaBiasMax = 1023;

struct LaArgs {
  int rows, vocab, requests, per_group;
  int chunk;   // tokens of a CTA in a pass, whole spans
  int passes;  // a power of two, as the CTAs of a cluster
  int vshift;  // log2 of both's product
  const void* x;
  void* y;
  long long x_stride, y_stride;
  int32_t* next;
  const int32_t *seq, *tokens, *tokens_len, *prompt_len, *draft, *row_start;
  long long tokens_stride;
  int tokens_base;
  const uint32_t* mask;
  int mask_words;
  const float *rep, *freq, *pres;
  const int32_t* bias_tokens;
  const float* bias;
  const int32_t* bias_len;
  int bias_stride;
  const uint32_t* allowed;
  long long allowed_stride;
  int allowed_rows;
  const int32_t* allowed_row;
  uint32_t* err;
};

// Bits whose unsigned order is the order of finite floats and infinities, both zeros alike; 0 is below all.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// 4 logits as they lie in memory; VEC: 16 (8) bytes at a time.
template <typename XT, bool VEC>
struct LaQuad {
  uint32_t w[sizeof(XT)];
  __device__ __forceinline__ void load(const XT* p, int n) {  // those past n: 0
    if constexpr (sizeof(XT) == 4) {
      if (VEC && n >= 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
      }
    } else {
      if (VEC && n >= 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(XT) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};

template <bool VEC>
__device__ __forceinline__ void la_store4(float* p, const float (&x)[4]) {
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = x[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void la_store4(uint16_t* p, const float (&x)[4]) {
  uint32_t h[2];
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(x[3]), "f"(x[2]));
  if (VEC) {
    *reinterpret_cast<uint2*>(p) = make_uint2(h[0], h[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ void la_store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void la_store1(uint16_t* p, float x) {
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(x));
  *p = static_cast<uint16_t>(h);
}

// What is known of a row of the group.
struct LaRow {
  int s;        // its request; -1: the row is left as it was
  int allowed;  // row of the masks of allowed tokens, -1: none
  int listed;   // its drafted tokens; more than kLaDrafts: not listed, counted in the words
  float rep, freq, pres;
};

// Grid: (CTAs of a cluster, groups of rows). Token numbers t are the CTA's own: v is
// (t / 512 * CTAs and passes + this one) * 512 + t % 512.
template <typename XT, typename YT, bool VEC>
__global__ void __launch_bounds__(kLaThreads, 2) logits_adjust_kernel(const LaArgs a) {
  extern __shared__ __align__(16) uint32_t s_word[];  // [chunk], then [kLaRows][chunk / 128] bits of quads with drafted tokens
  __shared__ unsigned long long s_best[kLaRows];
  __shared__ LaRow s_row[kLaRows];
  __shared__ int s_prompt[kLaRows];  // how many of the drafted tokens listed, the first ones, are the prompt's; not listed: those of rows before this
  __shared__ uint16_t s_draft[kLaRows][kLaDrafts], s_touched[kLaTouched];
  __shared__ uint32_t s_bits[kLaChunkMax / 32];  // tokens with a word
  __shared__ int s_count;                        // of them
  uint32_t* s_quad = s_word + a.chunk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = gridDim.x, rank = blockIdx.x, parts = a.chunk / 128;  // of 128 tokens: a warp's
  const int r0 = blockIdx.y * a.per_group, nrows = min(a.per_group, a.rows - r0);
  if (tid < kLaRows) s_best[tid] = 0;
  pdl_wait();
  pdl_trigger();
  for (int pass = 0; pass < a.passes; ++pass) {
    const int own = pass * ctas + rank, vmask = (1 << a.vshift) - 1;
    auto token_of = [&](int t) { return ((((t >> kLaSpan) << a.vshift) + own) << kLaSpan) + (t & ((1 << kLaSpan) - 1)); };
    // token v as the CTA numbers it, -1 if it is another one's or there is none
    auto local = [&](int v) -> int {
      if (v < 0 || v >= a.vocab || (v >> kLaSpan & vmask) != own) return -1;
      return (v >> kLaSpan >> a.vshift << kLaSpan) + (v & ((1 << kLaSpan) - 1));
    };
    // whether row number k of the request is on the way to row r
    auto on_way = [&](int r, int begin, int k) -> bool {
      return a.mask ? k < 32 * a.mask_words && (a.mask[static_cast<long long>(r) * a.mask_words + (k >> 5)] >> (k & 31) & 1u)
                    : k <= r - begin;
    };
    auto drafted = [&](int r, int begin, int k) -> int { return on_way(r, begin, k) ? local(a.draft[begin + k]) : -1; };
    // tokens of the request's text, as far as its arguments go
    auto text_len = [&](int s) -> long long { return a.tokens ? max(static_cast<long long>(a.tokens_len[s]) + a.tokens_base, 0ll) : 0; };
    auto drafts = [&](int s, int* begin) -> int {  // how many rows the request has, and its first
      *begin = a.row_start[s];
      return *begin < 0 ? 0 : min(kLaDraftMax, min(a.row_start[s + 1], a.rows) - *begin);
    };
    // ---- the rows: a warp each ----
    static_assert(kLaRows <= kLaWarps, "a warp for every row");
    if (warp < nrows) {
      const int r = r0 + warp, s = a.seq ? a.seq[r] : r;
      const bool live = s >= 0 && s < a.requests;
      for (int k = lane; k < parts; k += 32) s_quad[warp * parts + k] = 0;
      __syncwarp();
      int listed = 0, prompt = 0;
      if (live && a.draft) {
        int begin;
        const int rows = drafts(s, &begin);
        // drafted tokens on the way that are the prompt's: all in front of row `cut`
        const long long left = a.prompt_len ? a.prompt_len[s] - text_len(s) : 0;
        int cut = 0;
        if (left > 0) {
          long long before = 0;
          cut = 0x7fffffff;
          for (int k0 = 0; k0 < rows && before < left; k0 += 32) {
            const bool on = k0 + lane < rows && on_way(r, begin, k0 + lane);
            const unsigned way = __ballot_sync(0xffffffffu, on);
            if (before + __popc(way) >= left) {  // the one with number `left` is in this word
              const unsigned last = __ballot_sync(0xffffffffu, on && before + __popc(way & ((2u << lane) - 1u)) == left);
              cut = k0 + __ffs(last);
            }
            before += __popc(way);
          }
        }
        for (int k0 = 0; k0 < rows; k0 += 32) {
          const int t = k0 + lane < rows ? drafted(r, begin, k0 + lane) : -1;
          const unsigned hit = __ballot_sync(0xffffffffu, t >= 0);
          const int at = listed + __popc(hit & ((1u << lane) - 1u));
          if (t >= 0 && at < kLaDrafts) {
            s_draft[warp][at] = static_cast<uint16_t>(t);
            atomicOr(s_quad + warp * parts + (t >> 7), 1u << (t >> 2 & 31));
          }
          listed += __popc(hit);
          if (k0 < cut) prompt += __popc(cut - k0 < 32 ? hit & ((1u << (cut - k0)) - 1u) : hit);
        }
        if (listed > kLaDrafts) prompt = cut;
        if (listed > kLaDrafts) {
          __syncwarp();
          for (int k = lane; k < parts; k += 32) s_quad[warp * parts + k] = 0;
        }
      }
      if (lane == 0) {
        LaRow x;
        x.s = live ? s : -1;
        x.allowed = -1;
        x.listed = listed;
        s_prompt[warp] = prompt;
        x.rep = live && a.rep ? a.rep[s] : 1.f;
        x.freq = live && a.freq ? a.freq[s] : 0.f;
        x.pres = live && a.pres ? a.pres[s] : 0.f;
        if (live && a.allowed) {
          const int m = a.allowed_row ? a.allowed_row[r] : r;
          if (m >= 0 && m < a.allowed_rows)
            x.allowed = m;
          else if (m >= a.allowed_rows && rank == 0)
            atomicOr(a.err, ERR_BAD_TOKEN);
        }
        s_row[warp] = x;
      }
    }
    __syncthreads();
    // token t, whose word was `old`, has one now
    auto touch = [&](int t, uint32_t old) {
      if (old != 0 || (atomicOr(s_bits + (t >> 5), 1u << (t & 31)) >> (t & 31) & 1u)) return;
      const int at = atomicAdd(&s_count, 1);
      if (at < kLaTouched) s_touched[at] = static_cast<uint16_t>(t);
    };
    int built = -1;  // the request whose words are in place
    for (int i = 0; i < nrows; ++i) {
      const LaRow row = s_row[i];
      const int s = row.s, r = r0 + i;
      if (s < 0) continue;
      if (s != built) {
        __syncthreads();  // the rows before have been worked on
        for (int k = tid * 4; k < a.chunk; k += kLaThreads * 4) *reinterpret_cast<uint4*>(s_word + k) = make_uint4(0, 0, 0, 0);
        for (int k = tid; k < a.chunk / 32; k += kLaThreads) s_bits[k] = 0;
        if (tid == 0) s_count = 0;
        __syncthreads();
        if (a.tokens) {
          const int32_t* text = a.tokens + a.tokens_stride * s;
          const int held = static_cast<int>(min(text_len(s), min(static_cast<long long>(kLaTextMax), a.tokens_stride)));
          const int prompt = a.prompt_len ? a.prompt_len[s] : 0;
#pragma unroll 4
          for (int k = tid; k < held; k += kLaThreads) {
            const int t = local(text[k]);
            if (t < 0) continue;
            touch(t, k < prompt ? atomicOr(s_word + t, 0x80000000u) : atomicAdd(s_word + t, 1u));
          }
        }
        if (a.bias_tokens) {
          __syncthreads();  // the counts are whole: their bits do not change below
          const long long from = static_cast<long long>(a.bias_stride) * s;
          const int held = min(min(a.bias_len[s], a.bias_stride), kLaBiasMax);
          for (int k = tid; k < held; k += kLaThreads) {
            const int t = local(a.bias_tokens[from + k]);
            if (t < 0) continue;
            uint32_t old = s_word[t];
            while ((old >> 20 & 1023u) < static_cast<uint32_t>(k + 1)) {  // at most once for each bias of this token
              const uint32_t seen = atomicCAS(s_word + t, old, (old & ~(1023u << 20)) | static_cast<uint32_t>(k + 1) << 20);
              if (seen == old) break;
              old = seen;
            }
            touch(t, old);
          }
        }
        __syncthreads();
        built = s;
      }
      // more drafted tokens than a list holds go into the words and leave them again
      auto count = [&](bool in) {
        int begin;
        const int rows = drafts(s, &begin);
        __syncthreads();
        for (int k = tid; k < rows; k += kLaThreads) {
          const int t = drafted(r, begin, k);
          if (t < 0) continue;
          const uint32_t bit = 1u << 30;
          const uint32_t old = k >= s_prompt[i] ? atomicAdd(s_word + t, in ? 1u : 0xFFFFFFFFu) : in ? atomicOr(s_word + t, bit) : atomicAnd(s_word + t, ~bit);
          if (in) touch(t, old);
        }
        __syncthreads();
      };
      const bool spill = row.listed > kLaDrafts;
      const int listed = spill ? 0 : row.listed;
      if (spill) count(true);
      const uint32_t* ok = row.allowed >= 0 ? a.allowed + a.allowed_stride * row.allowed : nullptr;
      const XT* x = static_cast<const XT*>(a.x) + a.x_stride * r;
      YT* y = a.y ? static_cast<YT*>(a.y) + a.y_stride * r : nullptr;
      const uint32_t* quad = s_quad + i * parts;
      float best = -INFINITY;
      int best_v = 0;
      // ---- tokens without a rule but the mask: a warp's parts lie 16 apart, which are 4 spans ----
      static_assert(kLaWarps * 128 == 4 << kLaSpan, "a warp's next part");
      const int vocab = a.vocab, step = 4 << (kLaSpan + a.vshift), v_first = token_of(warp * 128 + lane * 4);
      const int shift = lane * 4 & 31;  // of the quad's bits in its word
      const uint32_t* with_word = s_bits + warp * 4 + (lane >> 3);
      const uint32_t* with_draft = s_quad + i * parts + warp;
#pragma unroll 1
      for (int v = v_first; v < vocab; v += kLaBatch * step) {
        LaQuad<XT, VEC> in[kLaBatch];
        uint32_t may[kLaBatch];
#pragma unroll
        for (int q = 0; q < kLaBatch; ++q)
          if (v + q * step < vocab) in[q].load(x + v + q * step, vocab - (v + q * step));
#pragma unroll
        for (int q = 0; q < kLaBatch; ++q) may[q] = 15u;
        if (ok) {
#pragma unroll
          for (int q = 0; q < kLaBatch; ++q)
            if (v + q * step < vocab) may[q] = ok[(v + q * step) >> 5] >> shift & 15u;
        }
#pragma unroll
        for (int q = 0; q < kLaBatch; ++q) {
          const int at = v + q * step;
          if (at >= vocab) break;
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = in[q].get(k);
          if (may[q] != 15u) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(may[q] >> k & 1u)) e[k] = -INFINITY;
          }
          uint32_t skip = with_word[q * 4 * kLaWarps] >> shift & 15u;
          if (with_draft[q * kLaWarps] >> lane & 1u) {
            const int t0 = ((with_draft - s_quad - i * parts) + q * kLaWarps) * 128 + lane * 4;
            for (int d = 0; d < listed; ++d) {
              const int t = s_draft[i][d] - t0;
              if (t >= 0 && t < 4) skip |= 1u << t;
            }
          }
          if (vocab - at < 4) skip |= 15u << (vocab - at) & 15u;
          if (skip == 0) {
            if (y) la_store4<VEC>(y + at, e);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (skip >> k & 1u)
                e[k] = -INFINITY;
              else if (y)
                la_store1(y + at + k, e[k]);
            }
          }
          const float top = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));  // (a NaN only of four)
          if (top > best) {  // (this thread's tokens rise: of equal ones the first stays)
            best = top;
            best_v = at + (e[0] == top ? 0 : e[1] == top ? 1 : e[2] == top ? 2 : 3);
          }
        }
        with_word += kLaBatch * 4 * kLaWarps;
        with_draft += kLaBatch * kLaWarps;
      }
      // ---- tokens with rules, one a thread ----
      auto rules = [&](int t, uint32_t w, uint32_t times) {
        const int v = token_of(t);
        LaQuad<XT, false> in;
        in.load(x + v, 1);
        float e = in.get(0);
        const uint32_t b = w >> 20 & 1023u;
        if (times || w >> 30) e = e > 0.f ? __fdiv_rn(e, row.rep) : __fmul_rn(e, row.rep);
        if (times) e = __fsub_rn(__fsub_rn(e, __fmul_rn(row.freq, static_cast<float>(times))), row.pres);
        if (b) e = __fadd_rn(e, a.bias[static_cast<long long>(a.bias_stride) * s + b - 1]);
        if (ok && !(ok[v >> 5] >> (v & 31) & 1u)) e = -INFINITY;
        if (y) la_store1(y + v, e);
        if (e > best || (e == best && best > -INFINITY && v < best_v)) best = e, best_v = v;
      };
      auto in_drafts = [&](int t) {
        if (!(quad[t >> 7] >> (t >> 2 & 31) & 1u)) return false;
        for (int d = 0; d < listed; ++d)
          if (s_draft[i][d] == t) return true;
        return false;
      };
      const int touched = s_count;
      if (touched <= kLaTouched) {
        for (int k = tid; k < touched; k += kLaThreads) {
          const int t = s_touched[k];
          if (!in_drafts(t)) rules(t, s_word[t], s_word[t] & 0xFFFFFu);
        }
      } else {
        for (int t = tid; t < a.chunk; t += kLaThreads)
          if ((s_bits[t >> 5] >> (t & 31) & 1u) && !in_drafts(t)) rules(t, s_word[t], s_word[t] & 0xFFFFFu);
      }
      for (int k = tid; k < listed; k += kLaThreads) {
        const int t = s_draft[i][k];
        uint32_t w = s_word[t], times = w & 0xFFFFFu;
        bool first = true;
        for (int d = 0; d < listed; ++d) {
          times += s_draft[i][d] == t && d >= s_prompt[i];
          first = first && (d >= k || s_draft[i][d] != t);
        }
        if (k < s_prompt[i]) w |= 1u << 30;  // (the first of equal ones stands for all)
        if (first) rules(t, w, times);
      }
      if (a.next) {
        unsigned long long key =
            best > -INFINITY ? static_cast<unsigned long long>(order_bits(best)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(best_v)) : 0ull;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
          if (other > key) key = other;
        }
        if (lane == 0 && key) atomicMax(s_best + i, key);
      }
      if (spill) count(false);
    }
    __syncthreads();
  }
  if (!a.next) return;
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && tid < nrows) {
    unsigned long long key = s_best[tid];
    for (int c = 1; c < ctas; ++c) {
      uint32_t at;
      unsigned long long other;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(s_best + tid)), "r"(c));
      asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(other) : "r"(at) : "memory");
      if (other > key) key = other;
    }
    const int r = r0 + tid, s = a.seq ? a.seq[r] : r;
    if (s >= 0 && s < a.requests) a.next[r] = key ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
  }
  // no CTA ends before the first has read its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename XT, typename YT, bool VEC>
cudaError_t la_launch_one(const LaArgs& a, int ctas, int groups, const DeviceInfo& di, cudaStream_t st) {
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    const cudaError_t e = allow_smem_shared(logits_adjust_kernel<XT, YT, VEC>, (kLaChunkMax + kLaRows * kLaChunkMax / 128) * 4);
    if (e != cudaSuccess) return e;
    lifted[di.device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, groups);
  cfg.blockDim = dim3(kLaThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.chunk + kLaRows * a.chunk / 128) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logits_adjust_kernel<XT, YT, VEC>, a);
}

template <typename XT, typename YT>
cudaError_t la_launch(const LaArgs& a, bool vec, int ctas, int groups, const DeviceInfo& di, cudaStream_t st) {
  return vec ? la_launch_one<XT, YT, true>(a, ctas, groups, di, st) : la_launch_one<XT, YT, false>(a, ctas, groups, di, st);
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" dec_status logits_adjust(const logits_adjust_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "logits_adjust: NULL arguments");
  auto type = [](int t) { return t == DEC_F32 || t == DEC_BF16; };
  if (a->rows < 0 || a->vocab < 1 || a->vocab > 1 << 20 || a->requests < 0 || !type(a->xdtype) || !type(a->ydtype) ||
      a->mask_words < 0 || a->mask_words > 1 << 20 || a->bias_stride < 0 || a->allowed_rows < 0 || a->tokens_base < 0)
    return fail(nullptr, DEC_EINVAL,
                "logits_adjust: rows %d, vocab %d, requests %d, xdtype %d, ydtype %d, mask_words %d, bias_stride %d, "
                "allowed_rows %d, tokens_base %d",
                a->rows, a->vocab, a->requests, a->xdtype, a->ydtype, a->mask_words, a->bias_stride, a->allowed_rows,
                a->tokens_base);
  if (a->rows == 0) return DEC_OK;
  if (!a->logits || (!a->out && !a->next)) return fail(nullptr, DEC_EINVAL, "logits_adjust: NULL logits, or neither out nor next");
  if ((a->tokens && !a->tokens_len) || (a->draft_tokens && !a->row_start) || (a->bias_tokens && (!a->bias || !a->bias_len)))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: NULL pointer");
  if (a->draft_tokens && a->mask && a->mask_words == 0) return fail(nullptr, DEC_EINVAL, "logits_adjust: a mask of 0 words");
  const long long words = (a->vocab + 31) / 32;
  if (a->rows > 1 && (a->logits_stride < a->vocab || (a->out && a->out_stride < a->vocab)))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: rows of %d logits overlap at strides %lld and %lld", a->vocab,
                static_cast<long long>(a->logits_stride), static_cast<long long>(a->out_stride));
  if ((a->tokens && a->tokens_stride < 0) || (a->allowed && a->allowed_stride < words))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: tokens_stride %lld, allowed_stride %lld",
                static_cast<long long>(a->tokens_stride), static_cast<long long>(a->allowed_stride));
  if (!aligned_to(elem_bytes(a->xdtype), a->logits) || !aligned_to(elem_bytes(a->ydtype), a->out) ||
      !aligned_to(4, a->next, a->seq, a->tokens, a->tokens_len, a->prompt_len, a->draft_tokens, a->row_start, a->mask,
                  a->repetition, a->frequency, a->presence, a->bias_tokens, a->bias, a->bias_len, a->allowed,
                  a->allowed_row))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: a pointer is not aligned to its elements");
  const bool in_place = a->out == a->logits;
  if (in_place && (a->xdtype != a->ydtype || (a->rows > 1 && a->logits_stride != a->out_stride)))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: out over logits needs their type and stride");
  const size_t rows = a->rows, n = a->requests;
  const Span in = span_rows(in_place ? nullptr : a->logits, a->rows, a->logits_stride, a->vocab, elem_bytes(a->xdtype));
  if (outputs_meet({span_rows(a->out, a->rows, a->out_stride, a->vocab, elem_bytes(a->ydtype)), {a->next, 4 * rows}},
                   {in, {a->seq, 4 * rows}, {a->tokens, 4 * n * static_cast<size_t>(a->tokens ? a->tokens_stride : 0)},
                    {a->tokens_len, 4 * n}, {a->prompt_len, 4 * n}, {a->draft_tokens, 4 * rows}, {a->row_start, 4 * (n + 1)},
                    {a->mask, 4 * rows * a->mask_words}, {a->repetition, 4 * n}, {a->frequency, 4 * n}, {a->presence, 4 * n},
                    {a->bias_tokens, 4 * n * a->bias_stride}, {a->bias, 4 * n * a->bias_stride}, {a->bias_len, 4 * n},
                    span_rows(a->allowed, a->allowed_rows, a->allowed_stride, words, 4), {a->allowed_row, 4 * rows}}))
    return fail(nullptr, DEC_EINVAL, "logits_adjust: an output overlaps another argument");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  LaArgs k{};
  k.rows = a->rows;
  k.vocab = a->vocab;
  k.requests = a->requests;
  k.x = a->logits;
  k.y = a->out;
  k.x_stride = a->logits_stride;
  k.y_stride = a->out_stride;
  k.next = a->next;
  k.seq = a->seq;
  k.tokens = a->tokens;
  k.tokens_len = a->tokens_len;
  k.prompt_len = a->prompt_len;
  k.tokens_stride = a->tokens_stride;
  k.tokens_base = a->tokens_base;
  k.draft = a->draft_tokens;
  k.row_start = a->row_start;
  k.mask = a->mask;
  k.mask_words = a->mask_words;
  k.rep = a->repetition;
  k.freq = a->frequency;
  k.pres = a->presence;
  k.bias_tokens = a->bias_tokens;
  k.bias = a->bias;
  k.bias_len = a->bias_len;
  k.bias_stride = a->bias_stride;
  k.allowed = a->allowed;
  k.allowed_stride = a->allowed_stride;
  k.allowed_rows = a->allowed_rows;
  k.allowed_row = a->allowed_row;
  auto quads = [](const void* p, long long stride, int dtype, int rows) {
    const size_t e = elem_bytes(dtype);
    return reinterpret_cast<uintptr_t>(p) % (4 * e) == 0 && (rows == 1 || stride % 4 == 0);
  };
  const bool vec = quads(a->logits, a->logits_stride, a->xdtype, a->rows) && (!a->out || quads(a->out, a->out_stride, a->ydtype, a->rows));
  k.err = di.err;
  // CTAs of a cluster: at least 2048 tokens each; passes over the vocabulary
  int ctas = kLaCluster;
  while (ctas > 1 && a->vocab < 2048 * ctas) ctas /= 2;
  const int spans = (a->vocab + (1 << kLaSpan) - 1) >> kLaSpan;
  auto chunk = [&](int parts) { return (spans + parts - 1) / parts << kLaSpan; };
  k.passes = 1;
  while (chunk(ctas * k.passes) > kLaChunkMax) k.passes *= 2;
  k.chunk = chunk(ctas * k.passes);
  while (1 << k.vshift < ctas * k.passes) ++k.vshift;
  // rows of a cluster: all clusters resident at once where that is not too many rows
  const int resident = 2 * di.sms / ctas;
  k.per_group = (a->rows + resident - 1) / resident;
  if (k.per_group > kLaRows) k.per_group = kLaRows;
  const long long groups = (static_cast<long long>(a->rows) + k.per_group - 1) / k.per_group;
  if (groups > 65535) return fail(nullptr, DEC_EINVAL, "logits_adjust: %d rows", a->rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int g = static_cast<int>(groups);
  const bool xf = a->xdtype == DEC_F32, yf = a->ydtype == DEC_F32;
  const cudaError_t e = xf ? (yf ? la_launch<float, float>(k, vec, ctas, g, di, s) : la_launch<float, uint16_t>(k, vec, ctas, g, di, s))
                           : (yf ? la_launch<uint16_t, float>(k, vec, ctas, g, di, s) : la_launch<uint16_t, uint16_t>(k, vec, ctas, g, di, s));
  WSG_CUDA_TRY(nullptr, e);
  return DEC_OK;
}
