// logits_adjust: penalties for repeated tokens, biases and masks of allowed tokens
// on the logits, and the greedy token of what results ("Megakernels", "GPU-wide
// end-to-end generation": greedy argmax on the GPU, lowest ID on ties).
//
// Mathematics, for token v of a row: x = x / rep or x * rep (v in the text), x - freq
// n(v), x - pres (n(v) > 0), x + bias, -inf (not allowed), each step rounded to
// float32 as the definition says.
//
// A cluster of CTAs takes a group of consecutive rows; each of its CTAs takes a range
// of the vocabulary, for which it keeps one word a token in shared memory: the times
// that the token came (bits 0-19), the number of its bias in the list (20-29) and
// whether the prompt has it (31). The words are built once a request from its text,
// by integer atomics whose order does not matter, and reused for all rows of it; a
// row's drafted tokens are added before it and taken away after it. So the logits
// are read and written once and nothing is kept between calls. The CTAs' best tokens,
// as (order-preserving bits of the value, inverted token), meet in the first CTA's
// shared memory.
//
// Bound by memory for many rows, by a chain of latencies (text, logits, cluster) for one.
#include "common.h"
#include "ptx.cuh"
#include "spans.h"

namespace wsg {
namespace {

constexpr int kLaThreads = 512, kLaCluster = 8, kLaChunkMax = 24576, kLaRows = 32;
constexpr int kLaTextMax = 1 << 19, kLaDraftMax = (1 << 19) - 1, kLaBiasMax = 1023;

struct LaArgs {
  int rows, vocab, requests, per_group, chunk, passes;
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
  int vec;  // 4 elements at a time
  uint32_t* err;
};

// Bits whose unsigned order is the order of finite floats and infinities; 0 is below all.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

template <typename XT>
__device__ __forceinline__ void la_load4(const XT* p, bool vec, int n, float (&x)[4]) {
  if constexpr (sizeof(XT) == 4) {
    if (vec && n >= 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = i < n ? p[i] : 0.f;
    }
  } else {
    if (vec && n >= 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
    }
  }
}

template <typename YT>
__device__ __forceinline__ void la_store4(YT* p, bool vec, int n, const float (&x)[4]) {
  if constexpr (sizeof(YT) == 4) {
    if (vec && n >= 4) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = x[i];
    }
  } else {
    uint32_t h[2];
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(x[3]), "f"(x[2]));
    if (vec && n >= 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(h[0], h[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Grid: (CTAs of a cluster, groups of rows).
template <typename XT, typename YT>
__global__ void __launch_bounds__(kLaThreads, 2) logits_adjust_kernel(const LaArgs a) {
  extern __shared__ __align__(16) uint32_t s_word[];  // [chunk]
  __shared__ unsigned long long s_best[kLaRows];
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = gridDim.x, rank = blockIdx.x;
  const int r0 = blockIdx.y * a.per_group, nrows = min(a.per_group, a.rows - r0);
  if (tid < kLaRows) s_best[tid] = 0;
  pdl_wait();
  pdl_trigger();
  for (int pass = 0; pass < a.passes; ++pass) {
    const int v0 = (pass * ctas + rank) * a.chunk, n = min(a.chunk, a.vocab - v0);
    if (n <= 0) break;  // (the CTAs after this one have nothing either)
    int built = -1;     // the request whose words are in place
    for (int i = 0; i < nrows; ++i) {
      const int r = r0 + i, s = a.seq ? a.seq[r] : r;
      if (s < 0 || s >= a.requests) continue;
      if (s != built) {
        __syncthreads();
        for (int k = tid * 4; k < a.chunk; k += kLaThreads * 4) *reinterpret_cast<uint4*>(s_word + k) = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (a.tokens) {
          const int32_t* text = a.tokens + a.tokens_stride * s;
          const long long len = static_cast<long long>(a.tokens_len[s]) + a.tokens_base;
          const int count = static_cast<int>(min(max(len, 0ll), min(static_cast<long long>(kLaTextMax), a.tokens_stride)));
          const int prompt = a.prompt_len ? a.prompt_len[s] : 0;
#pragma unroll 4
          for (int k = tid; k < count; k += kLaThreads) {
            const long long t = static_cast<long long>(text[k]) - v0;
            if (t >= 0 && t < n) {
              if (k < prompt)
                atomicOr(s_word + t, 0x80000000u);
              else
                atomicAdd(s_word + t, 1u);
            }
          }
        }
        if (a.bias_tokens) {
          __syncthreads();  // the counts are whole: their bits do not change below
          const long long at = static_cast<long long>(a.bias_stride) * s;
          const int count = min(min(a.bias_len[s], a.bias_stride), kLaBiasMax);
          for (int k = tid; k < count; k += kLaThreads) {
            const long long t = static_cast<long long>(a.bias_tokens[at + k]) - v0;
            if (t < 0 || t >= n) continue;
            uint32_t old = s_word[t];
            while ((old >> 20 & 1023u) < static_cast<uint32_t>(k + 1)) {  // at most once for each bias of this token
              const uint32_t seen = atomicCAS(s_word + t, old, (old & ~(1023u << 20)) | static_cast<uint32_t>(k + 1) << 20);
              if (seen == old) break;
              old = seen;
            }
          }
        }
        built = s;
      }
      // the drafted tokens on the way to this row, added (+1) or taken away (-1)
      auto drafted = [&](uint32_t d) {
        const int begin = a.row_start[s], rows = min(a.row_start[s + 1], a.rows) - begin;
        const int own = r - begin, most = min(kLaDraftMax, a.mask ? min(rows, 32 * a.mask_words) : min(rows, own + 1));
        if (begin < 0) return;
        for (int k = tid; k < most; k += kLaThreads) {
          if (a.mask && !(a.mask[static_cast<long long>(r) * a.mask_words + (k >> 5)] >> (k & 31) & 1u)) continue;
          const long long t = static_cast<long long>(a.draft[begin + k]) - v0;
          if (t >= 0 && t < n) atomicAdd(s_word + t, d);
        }
      };
      if (a.draft) {
        __syncthreads();
        drafted(1u);
      }
      __syncthreads();
      const float rep = a.rep ? a.rep[s] : 1.f, freq = a.freq ? a.freq[s] : 0.f, pres = a.pres ? a.pres[s] : 0.f;
      const uint32_t* ok = nullptr;
      if (a.allowed) {
        const int m = a.allowed_row ? a.allowed_row[r] : r;
        if (m >= 0 && m < a.allowed_rows)
          ok = a.allowed + a.allowed_stride * m;
        else if (m >= a.allowed_rows && tid == 0 && rank == 0)
          atomicOr(a.err, ERR_BAD_TOKEN);
      }
      const XT* x = static_cast<const XT*>(a.x) + a.x_stride * r + v0;
      YT* y = a.y ? static_cast<YT*>(a.y) + a.y_stride * r + v0 : nullptr;
      float best = -INFINITY;
      int best_v = 0;
#pragma unroll 4
      for (int k = tid * 4; k < n; k += kLaThreads * 4) {
        float e[4];
        la_load4(x + k, a.vec, n - k, e);
        const uint4 w4 = *reinterpret_cast<const uint4*>(s_word + k);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        const uint32_t bits = ok ? ok[(v0 + k) >> 5] >> ((v0 + k) & 31) : 15u;  // (4 divides the chunks)
        if (w4.x | w4.y | w4.z | w4.w) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t times = w[j] & 0xFFFFFu, b = w[j] >> 20 & 1023u;
            if (times || w[j] >> 31) e[j] = e[j] > 0.f ? __fdiv_rn(e[j], rep) : __fmul_rn(e[j], rep);
            if (times) e[j] = __fsub_rn(__fsub_rn(e[j], __fmul_rn(freq, static_cast<float>(times))), pres);
            if (b) e[j] = __fadd_rn(e[j], a.bias[static_cast<long long>(a.bias_stride) * s + b - 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!(bits >> j & 1u)) e[j] = -INFINITY;
          if (k + j < n && e[j] > best) best = e[j], best_v = v0 + k + j;
        }
        if (y) la_store4(y + k, a.vec, n - k, e);
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
      if (a.draft) {
        __syncthreads();
        drafted(0xFFFFFFFFu);
      }
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

template <typename XT, typename YT>
cudaError_t la_launch(const LaArgs& a, int ctas, int groups, const DeviceInfo& di, cudaStream_t st) {
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    const cudaError_t e = allow_smem(logits_adjust_kernel<XT, YT>, kLaChunkMax * 4);
    if (e != cudaSuccess) return e;
    lifted[di.device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, groups);
  cfg.blockDim = dim3(kLaThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.chunk) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logits_adjust_kernel<XT, YT>, a);
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
  k.vec = quads(a->logits, a->logits_stride, a->xdtype, a->rows) && (!a->out || quads(a->out, a->out_stride, a->ydtype, a->rows));
  k.err = di.err;
  // CTAs of a cluster: at least 2048 tokens each; their chunks, in whole words of a mask
  int ctas = kLaCluster;
  while (ctas > 1 && a->vocab < 2048 * ctas) ctas /= 2;
  const int share = (a->vocab + ctas - 1) / ctas;
  k.passes = (share + kLaChunkMax - 1) / kLaChunkMax;
  k.chunk = ((share + k.passes - 1) / k.passes + 127) / 128 * 128;
  // rows of a cluster: all clusters resident at once where that is not too many rows
  const int resident = 2 * di.sms / ctas;
  k.per_group = (a->rows + resident - 1) / resident;
  if (k.per_group > kLaRows) k.per_group = kLaRows;
  const long long groups = (static_cast<long long>(a->rows) + k.per_group - 1) / k.per_group;
  if (groups > 65535) return fail(nullptr, DEC_EINVAL, "logits_adjust: %d rows", a->rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int g = static_cast<int>(groups);
  const bool xf = a->xdtype == DEC_F32, yf = a->ydtype == DEC_F32;
  const cudaError_t e = xf ? (yf ? la_launch<float, float>(k, ctas, g, di, s) : la_launch<float, uint16_t>(k, ctas, g, di, s))
                           : (yf ? la_launch<uint16_t, float>(k, ctas, g, di, s) : la_launch<uint16_t, uint16_t>(k, ctas, g, di, s));
  WSG_CUDA_TRY(nullptr, e);
  return DEC_OK;
}
