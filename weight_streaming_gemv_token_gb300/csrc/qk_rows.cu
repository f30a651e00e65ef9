// qk_norm_rope and kv_append_paged: per-head RMS norm of queries and keys with
// the position rotation in the same pass, and the store of keys and values
// into pages ("Megakernels", "What runs in the DSL": per-head Q/K RMSNorm,
// RoPE, KV update).
//
// Mathematics: y = x / sqrt(mean(x^2) + eps) * g per head; the pair (a, b) at
// angle t becomes (a cos t - b sin t, a sin t + b cos t), t = position * w_i.
// The angle is kept in turns as a 64-bit fixed-point fraction, F_i = frac(w_i /
// 2 pi) * 2^64: position * F_i modulo 2^64 is the exact fraction of a turn for
// that F_i, by integer multiplication, and nothing runs on the slow double pipe. F_i
// is w_i / 2 pi to 2^-64 of a turn (fewer bits than w_i has where that is small), which
// the farthest position makes 2^-33. The top 32 bits go to sincospif.
//
// Layout: a unit of lanes holds one head, 8 consecutive elements a lane (one
// 16-byte load of bfloat16, two of float32), and walks several heads of a row so
// that the row's cosines and sines are computed once and stay in registers.
// The half layout pairs element i with i + rot / 2, which another lane of the
// unit holds (a shuffle); interleaved pairs lie inside a lane; partners that
// straddle lanes go through shared memory. Each element is read and written once:
// bound by memory for many rows, by latency for few. Measured with 16 + 8 heads of
// 128: 1 row 3 us; 8,191 rows float32 36 us (5.6 TB/s), bfloat16 with half of each
// head rotated 25 us (4.0 TB/s; the same without norm and rotation 18).
#include <cmath>

#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {
namespace {

constexpr int kRowsThreads = 256;
struct QkRowsArgs {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;  // k_out, v_out: rows, or the pools
  long long q_stride, k_stride, v_stride, qo_stride, ko_stride;
  const float *g_q, *g_k;
  const int32_t* pos;
  const double* inv_freq;
  float eps, factor;
  int rows, n_q, n_kv, d, rot, interleaved;
  int per_unit;             // heads a unit walks
  int q_groups, kv_groups;  // groups of that many query and key (or value) heads
  int vec_x, vec_y;  // 16-byte accesses possible
  int y_f32, kv_f32;  // type of q_out (and k_out of qk_norm_rope), of the pools
  int paged;
  PagePool pool;
  const int32_t* table;
  const int32_t* seq;
  int n_seq, base_pos;
  uint32_t* err;
};

// Two floats as packed bfloat16 (low half: x), rounded to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  return h;
}

// 8 elements to float32 or bfloat16 memory, rounded once.
__device__ __forceinline__ void put8(void* base, long long at, int f32, int vec, const float (&x)[8]) {
  if (f32) {
    float* p = static_cast<float*>(base) + at;
    if (vec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = x[e];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack2(x[2 * e], x[2 * e + 1]);
    if (vec) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// frac(w / 2 pi) * 2^64 for w in radians, in integers: |w| = M 2^(E - 63) with a
// 64-bit M, 1 / 2 pi = C 2^-66, so the product is (M C) 2^(E - 129).
__device__ __forceinline__ unsigned long long turns64(double w) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(w));
  const int E = static_cast<int>((bits >> 52) & 0x7FFu) - 1023;
  const unsigned long long M = (bits << 11) | 0x8000000000000000ull, C = 0xA2F9836E4E441529ull;  // 2 / pi * 2^64
  const unsigned long long hi = __umul64hi(M, C), lo = M * C;
  unsigned long long f;  // floor(M C 2^(E - 65)) mod 2^64
  if (E <= 1)
    f = E > -63 ? hi >> (1 - E) : 0;
  else if (E <= 64)
    f = (hi << (E - 1)) | (lo >> (65 - E));
  else
    f = 0;  // beyond 2^65 radians a position the double itself holds no fraction of a turn
  return static_cast<long long>(bits) < 0 ? 0ull - f : f;
}

// Cosine and sine at a position, f the turns per position as turns64 gives them.
__device__ __forceinline__ void turn(unsigned long long f, uint32_t pos, float factor, float* c, float* s) {
  const int32_t t = static_cast<int32_t>(static_cast<uint32_t>((f * pos) >> 32));
  sincospif(static_cast<float>(t) * 0x1p-31f, s, c);  // in half turns
  *c *= factor;
  *s *= factor;
}

// 8 elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) == 4 ? 2 : 1];
};

template <typename T>
__device__ __forceinline__ Raw8<T> fetch8(const T* p, bool vec) {
  Raw8<T> r;
  if (vec) {
    r.w[0] = reinterpret_cast<const uint4*>(p)[0];
    if constexpr (sizeof(T) == 4) r.w[1] = reinterpret_cast<const uint4*>(p)[1];
  } else {
    uint32_t v[4 * sizeof(r.w) / sizeof(uint4)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v) / 4); ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = __float_as_uint(p[i]);
      else
        v[i] = p[2 * i] | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
    }
    r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if constexpr (sizeof(T) == 4) r.w[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&x)[8]) {
  const uint32_t a[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
  if constexpr (sizeof(T) == 4) {
    const uint32_t b[4] = {r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(a[e]), x[4 + e] = __uint_as_float(b[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(a[e] << 16), x[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
  }
}

// Pairs of floats for the two-wide float32 instructions.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ void unpair(Pair p, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(p));
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// How a head's pairs lie in its lanes.
enum PairMode : int {
  PAIR_LANES = 0,   // half layout, rot / 2 a multiple of 8: whole lanes are partners
  PAIR_INSIDE = 1,  // interleaved, rot a multiple of 8: inside a lane
  PAIR_STAGED = 2   // any other: through shared memory, decided for each element
};

// A unit of LPH lanes (a power of two, 8 LPH >= d) walks rows; blockIdx.y is a
// group of up to per_unit heads of one kind (queries, keys, values in turn), so
// that what depends on the kind is settled once. The next batch of heads is
// always on its way while one is worked on, across rows too.
template <typename XT, int LPH, int MODE, bool VEC>
__global__ void __launch_bounds__(kRowsThreads, 3) qk_rows_kernel(const QkRowsArgs a) {
  constexpr int kBatch = sizeof(XT) == 4 ? 2 : 4;  // heads a batch
  __shared__ float stage[MODE == PAIR_STAGED ? kRowsThreads * 8 : 1];
  const int tid = threadIdx.x, li = tid % LPH, e0 = li * 8;
  const int half = a.rot >> 1;
  int group = blockIdx.y, kind = 0;
  if (group >= a.q_groups) group -= a.q_groups, kind = 1;
  if (kind == 1 && group >= a.kv_groups) group -= a.kv_groups, kind = 2;
  const int h0 = group * a.per_unit, n = min(a.per_unit, (kind == 0 ? a.n_q : a.n_kv) - h0);
  const XT* in = static_cast<const XT*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + h0 * a.d + e0;
  const long long in_stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
  void* out = kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out;
  const bool pool = kind > 0 && a.paged;
  const int out_f32 = pool ? a.kv_f32 : a.y_f32, vec_out = VEC || pool;
  const float* g = kind == 0 ? a.g_q : kind == 1 ? a.g_k : nullptr;
  const int mate = (tid & 31) + (e0 >= a.rot ? 0 : e0 < half ? half >> 3 : -(half >> 3));  // PAIR_LANES
  // register e & 1 of pair e / 2 holds element el(e) of the lane: partners lie in the
  // same places of neighbouring pairs where they are inside the lane
  auto el = [](int e) { return MODE == PAIR_INSIDE ? (e & 4) + ((e >> 1) & 1) + 2 * (e & 1) : e; };
  // the element that partners element e
  auto partner = [&](int e) { return e >= a.rot ? e : a.interleaved ? e ^ 1 : e < half ? e + half : e - half; };
  const float mean = 1.f / static_cast<float>(a.d);

  // (a padded row's elements are read for nothing)
  Raw8<XT> next[kBatch];
  auto fetch = [&](long long r, int b0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      next[i] = r < a.rows && b0 + i < n && e0 < a.d ? fetch8(in + in_stride * r + (b0 + i) * a.d, VEC) : Raw8<XT>{};
  };
  long long r = static_cast<long long>(blockIdx.x) * (kRowsThreads / LPH) + tid / LPH;
  const long long rstep = static_cast<long long>(gridDim.x) * (kRowsThreads / LPH);
  pdl_wait();  // inputs come from the stream's previous kernel
  pdl_trigger();
  fetch(r, 0);
  // the gains, and the turns per position of the pairs this lane computes
  __shared__ __align__(16) float s_gain[128];
  if (g) {
    for (int i = tid; i < a.d; i += kRowsThreads) s_gain[i] = g[i];
  }
  constexpr int NF = MODE == PAIR_STAGED ? 8 : 4;
  unsigned long long turns[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int e = e0 + j;
    int i;
    if (MODE == PAIR_INSIDE) i = e0 / 2 + j;
    else if (MODE == PAIR_LANES) i = e0 >= half ? e - half + 4 : e;  // a lane and its mate: four pairs each
    else i = a.interleaved ? e >> 1 : e >= half ? e - half : e;
    turns[j] = kind < 2 && (MODE == PAIR_STAGED ? e : e0) < a.rot ? turns64(a.inv_freq[i]) : 0;
  }
  __syncthreads();
  int pos_next = r < a.rows ? a.pos[r] : -1;
  // the trip count is the CTA's: its first unit's rows
  for (long long rc = static_cast<long long>(blockIdx.x) * (kRowsThreads / LPH); rc < a.rows; rc += rstep, r += rstep) {
    const int pos = pos_next;
    const bool live = pos >= 0 && e0 < a.d;
    pos_next = r + rstep < a.rows ? a.pos[r + rstep] : -1;

    // where this row's heads go: element e0 of head h0, and from head to head
    long long to = (kind == 0 ? a.qo_stride : a.ko_stride) * r + h0 * a.d + e0, step = a.d;
    bool stores = live;
    if (pool && live) {
      const int s = a.seq ? a.seq[r] : static_cast<int>(r);
      const long long idx = static_cast<long long>(pos) - a.base_pos;
      const int page = s >= 0 && s < a.n_seq ? page_of(a.pool, a.table + static_cast<long long>(s) * a.pool.width, idx) : -1;
      stores = page >= 0;
      if (stores) {
        to = pool_row(a.pool, page, h0, idx) * a.d + e0;
        step = static_cast<long long>(a.d) << a.pool.shift;
      } else if (li == 0) {
        atomicOr(a.err, ERR_BAD_PAGE);
      }
    }

    // element e of this lane: y = (x * cg + partner * sg) / rms with the gains of
    // both and the sign in cg and sg; lanes that are not turned only scale
    const bool turned = kind < 2 && live && e0 < a.rot;  // PAIR_STAGED: some of the elements
    float cg[8], sg[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cg[e] = 1.f, sg[e] = 0.f;
    if (kind < 2 && a.rot > 0) {
      if (MODE == PAIR_INSIDE) {
        if (turned) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float c, s;
            turn(turns[j], static_cast<uint32_t>(pos), a.factor, &c, &s);
            cg[2 * j] = cg[2 * j + 1] = c;
            sg[2 * j] = -s, sg[2 * j + 1] = s;
          }
        }
      } else if (MODE == PAIR_LANES) {
        // a lane and its mate turn the same 8 pairs: each computes four of them
        const bool upper = e0 >= half;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float c = 1.f, s = 0.f;
          if (turned) turn(turns[j], static_cast<uint32_t>(pos), a.factor, &c, &s);
          const float c2 = __shfl_sync(0xffffffffu, c, mate), s2 = __shfl_sync(0xffffffffu, s, mate);
          cg[j] = upper ? c2 : c;
          cg[j + 4] = upper ? c : c2;
          sg[j] = upper ? s2 : -s;
          sg[j + 4] = upper ? s : -s2;
        }
      } else if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          const bool upper = a.interleaved ? e & 1 : e >= half;
          if (e >= a.rot) continue;
          float c, s;
          turn(turns[j], static_cast<uint32_t>(pos), a.factor, &c, &s);
          cg[j] = c;
          sg[j] = upper ? s : -s;
        }
      }
    }
    if (g && e0 < a.d) {
      float ga[8], gm[8];  // of the lane's elements, of their partners
      const int m0 = MODE == PAIR_LANES && turned ? (e0 < half ? e0 + half : e0 - half) : e0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 u = *reinterpret_cast<const float4*>(s_gain + e0 + 4 * q);
        const float4 w = *reinterpret_cast<const float4*>(s_gain + m0 + 4 * q);
        ga[4 * q] = u.x, ga[4 * q + 1] = u.y, ga[4 * q + 2] = u.z, ga[4 * q + 3] = u.w;
        gm[4 * q] = w.x, gm[4 * q + 1] = w.y, gm[4 * q + 2] = w.z, gm[4 * q + 3] = w.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cg[j] *= ga[j];
        sg[j] *= MODE == PAIR_INSIDE ? ga[j ^ 1] : MODE == PAIR_LANES ? gm[j] : s_gain[turned ? partner(e0 + j) : e0];
      }
    }
    Pair cg2[4], sg2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cg2[j] = pair(cg[el(2 * j)], cg[el(2 * j + 1)]);
      sg2[j] = pair(sg[el(2 * j)], sg[el(2 * j + 1)]);
    }

    for (int b0 = 0; b0 < n; b0 += kBatch) {
      Raw8<XT> raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) raw[i] = next[i];
      if (b0 + kBatch < n)
        fetch(r, b0 + kBatch);
      else
        fetch(r + rstep, 0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[8];
        widen8(raw[i], x);
        if (kind < 2) {
          Pair v[4], p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = pair(x[el(2 * e)], x[el(2 * e + 1)]);
          float inv = 1.f;
          if (g) {
            const Pair s2 = fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0]))));
            float s0, s1;
            unpair(s2, &s0, &s1);
            float ss = s0 + s1;
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            // 1 / sqrt by the approximation and one Newton step
            const float t = fmaf(ss, mean, a.eps);
            inv = rsqrtf(t);
            if (t > 0.f && t < INFINITY) inv = fmaf(0.5f * inv, fmaf(-t * inv, inv, 1.f), inv);
          }
          if (MODE == PAIR_INSIDE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = v[e ^ 1];
          } else if (MODE == PAIR_LANES) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = pair(__shfl_sync(0xffffffffu, x[2 * e], mate), __shfl_sync(0xffffffffu, x[2 * e + 1], mate));
          } else {
            float* st = stage + (tid - li) * 8;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) st[e0 + e] = x[e];
            __syncwarp();
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = e0 + e < a.rot ? st[partner(e0 + e)] : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pair(q[2 * e], q[2 * e + 1]);
          }
          if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fma2(p[e], sg2[e], mul2(v[e], cg2[e]));
          } else if (g) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], cg2[e]);
          }
          if (g) {
            const Pair i2 = pair(inv, inv);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], i2);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) unpair(v[e], &x[el(2 * e)], &x[el(2 * e + 1)]);
        }
        if (stores && b0 + i < n) put8(out, to + (b0 + i) * step, out_f32, vec_out, x);
      }
    }
  }
}

template <typename XT, int LPH>
cudaError_t launch_mode(const QkRowsArgs& a, int sms, cudaStream_t st) {
  constexpr int kUnits = kRowsThreads / LPH;
  const long long blocks = (a.rows + static_cast<long long>(kUnits) - 1) / kUnits;
  const int groups = a.q_groups + (a.paged ? 2 : 1) * a.kv_groups;
  // three CTAs an SM; each walks the same number of rows
  const long long most = (3ll * sms + groups - 1) / groups, turns = (blocks + most - 1) / most;
  const dim3 grid(static_cast<unsigned>((blocks + turns - 1) / turns), static_cast<unsigned>(groups));
  const dim3 block(kRowsThreads);
  const bool vec = a.vec_x && a.vec_y;
  if (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0) {
    if (a.interleaved)
      return vec ? launch_k(qk_rows_kernel<XT, LPH, PAIR_INSIDE, true>, grid, block, 0, st, true, a)
                 : launch_k(qk_rows_kernel<XT, LPH, PAIR_INSIDE, false>, grid, block, 0, st, true, a);
    return vec ? launch_k(qk_rows_kernel<XT, LPH, PAIR_LANES, true>, grid, block, 0, st, true, a)
               : launch_k(qk_rows_kernel<XT, LPH, PAIR_LANES, false>, grid, block, 0, st, true, a);
  }
  return vec ? launch_k(qk_rows_kernel<XT, LPH, PAIR_STAGED, true>, grid, block, 0, st, true, a)
             : launch_k(qk_rows_kernel<XT, LPH, PAIR_STAGED, false>, grid, block, 0, st, true, a);
}

template <typename XT>
cudaError_t launch_rows(const QkRowsArgs& a, int lph, int sms, cudaStream_t st) {
  return lph == 2   ? launch_mode<XT, 2>(a, sms, st)
         : lph == 8 ? launch_mode<XT, 8>(a, sms, st)
                    : launch_mode<XT, 16>(a, sms, st);
}

bool is_float(int t) { return t == DEC_F32 || t == DEC_BF16; }

// Whether rows at p with a stride in elements can be read or written in 16-byte pieces.
bool pieces16(const void* p, long long stride, int dtype) {
  return aligned16(p) && stride * (dtype == DEC_F32 ? 4 : 2) % 16 == 0;
}

// Whether rows may go from `in` to `out`: over themselves only where every row stays in
// its place, or a unit writes over rows that others have yet to read.
bool in_place_ok(const void* in, const void* out, int rows, int xd, int yd, int64_t in_stride, int64_t out_stride) {
  return in != out || (xd == yd && (rows == 1 || in_stride == out_stride));
}

// Checks common to both calls, on the fields they share.
template <typename A>
dec_status check_rows(const A* a, const char* who) {
  if (a->rows < 0 || a->n_q < 0 || a->n_kv < 0 || a->n_q > 16384 || a->n_kv > 16384)
    return fail(nullptr, DEC_EINVAL, "%s: rows %d, n_q %d, n_kv %d", who, a->rows, a->n_q, a->n_kv);
  if (a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8)
    return fail(nullptr, DEC_EINVAL, "%s: head_dim must be a multiple of 8 up to 128, got %d", who, a->head_dim);
  if (!is_float(a->xdtype) || !is_float(a->ydtype))
    return fail(nullptr, DEC_EINVAL, "%s: xdtype %d, ydtype %d", who, a->xdtype, a->ydtype);
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2)
    return fail(nullptr, DEC_EINVAL, "%s: rot_dim must be even and at most head_dim, got %d", who, a->rot_dim);
  if (!(a->eps >= 0.f)) return fail(nullptr, DEC_EINVAL, "%s: eps must be >= 0", who);
  if (a->rows == 0) return DEC_OK;
  if (!a->positions || (a->n_q > 0 && (!a->q || !a->q_out)) || (a->n_kv > 0 && !a->k) ||
      (a->rot_dim > 0 && !a->inv_freq))
    return fail(nullptr, DEC_EINVAL, "%s: NULL pointer", who);
  if ((a->n_q > 0 && !(aligned_to(elem_bytes(a->xdtype), a->q) && aligned_to(elem_bytes(a->ydtype), a->q_out) &&
                       aligned_to(4, a->g_q))) ||
      (a->n_kv > 0 && !(aligned_to(elem_bytes(a->xdtype), a->k) && aligned_to(4, a->g_k))) ||
      !aligned_to(4, a->positions) || (a->rot_dim > 0 && !aligned_to(8, a->inv_freq)))
    return fail(nullptr, DEC_EINVAL, "%s: a pointer is not aligned to its elements", who);
  if (a->q_stride < 0 || a->k_stride < 0) return fail(nullptr, DEC_EINVAL, "%s: negative row stride", who);
  if (a->rows > 1 && a->n_q > 0 && a->q_out_stride < static_cast<long long>(a->n_q) * a->head_dim)
    return fail(nullptr, DEC_EINVAL, "%s: q_out rows overlap at stride %lld", who,
                static_cast<long long>(a->q_out_stride));
  return DEC_OK;
}

template <typename A>
QkRowsArgs shared_fields(const A* a) {
  QkRowsArgs k{};
  k.q = a->q;
  k.k = a->k;
  k.q_out = a->q_out;
  k.q_stride = a->q_stride;
  k.k_stride = a->k_stride;
  k.qo_stride = a->q_out_stride;
  k.g_q = a->g_q;
  k.g_k = a->g_k;
  k.pos = a->positions;
  k.inv_freq = a->inv_freq;
  k.eps = a->eps;
  k.factor = a->rope_factor;
  k.rows = a->rows;
  k.n_q = a->n_q;
  k.n_kv = a->n_kv;
  k.d = a->head_dim;
  k.rot = a->rot_dim;
  k.interleaved = a->interleaved != 0;
  k.y_f32 = a->ydtype == DEC_F32;
  k.vec_x = (a->n_q == 0 || pieces16(a->q, a->q_stride, a->xdtype)) && (a->n_kv == 0 || pieces16(a->k, a->k_stride, a->xdtype));
  k.vec_y = a->n_q == 0 || pieces16(a->q_out, a->q_out_stride, a->ydtype);
  return k;
}

dec_status run_rows(QkRowsArgs& k, int xd, const DeviceInfo& di, cudaStream_t st) {
  const int lph = k.d <= 16 ? 2 : k.d <= 64 ? 8 : 16;  // lanes of a unit
  // Heads a unit walks: more share the row's angles, fewer give more units.
  auto groups = [&](int per) {
    return static_cast<long long>(k.n_q + per - 1) / per + (k.paged ? 2 : 1) * static_cast<long long>((k.n_kv + per - 1) / per);
  };
  k.per_unit = 1;
  while (k.per_unit < 8 && k.rows * groups(2 * k.per_unit) * lph >= 3ll * kRowsThreads * di.sms) k.per_unit *= 2;
  k.q_groups = (k.n_q + k.per_unit - 1) / k.per_unit;
  k.kv_groups = (k.n_kv + k.per_unit - 1) / k.per_unit;
  WSG_CUDA_TRY(nullptr, xd == DEC_F32 ? launch_rows<float>(k, lph, di.sms, st) : launch_rows<uint16_t>(k, lph, di.sms, st));
  return DEC_OK;
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" dec_status rope_frequencies(const rope_scaling* s, double* h_inv_freq, float* h_factor) {
  if (!s || !h_inv_freq || !h_factor) return fail(nullptr, DEC_EINVAL, "rope_frequencies: NULL pointer");
  if (s->rot_dim < 2 || s->rot_dim > 128 || s->rot_dim % 2)
    return fail(nullptr, DEC_EINVAL, "rope_frequencies: rot_dim must be even, 2..128, got %d", s->rot_dim);
  if (!(s->theta > 0.0) || !std::isfinite(s->theta)) return fail(nullptr, DEC_EINVAL, "rope_frequencies: theta must be positive");
  if (s->kind < ROPE_PLAIN || s->kind > ROPE_RAMP) return fail(nullptr, DEC_EINVAL, "rope_frequencies: kind %d", s->kind);
  if (s->kind != ROPE_PLAIN && !(s->factor >= 1.0 && std::isfinite(s->factor)))
    return fail(nullptr, DEC_EINVAL, "rope_frequencies: factor must be at least 1");
  if (s->kind == ROPE_BASE && s->rot_dim < 4)
    return fail(nullptr, DEC_EINVAL, "rope_frequencies: ROPE_BASE needs rot_dim >= 4");
  if (s->kind == ROPE_RAMP &&
      !(s->orig_context > 0.0 && s->beta_slow > 0.0 && s->beta_fast > s->beta_slow && std::isfinite(s->beta_fast)))
    return fail(nullptr, DEC_EINVAL, "rope_frequencies: ROPE_RAMP needs orig_context > 0 and 0 < beta_slow < beta_fast");
  const double rot = s->rot_dim;
  const double base = s->kind == ROPE_BASE ? s->theta * std::pow(s->factor, rot / (rot - 2.0)) : s->theta;
  for (int i = 0; i < s->rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot);
    if (s->kind == ROPE_LINEAR) w /= s->factor;
    if (s->kind == ROPE_RAMP) {
      const double turns = s->orig_context * w / 6.283185307179586;
      double keep = (turns - s->beta_slow) / (s->beta_fast - s->beta_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      w = w * keep + w / s->factor * (1.0 - keep);
    }
    h_inv_freq[i] = w;
  }
  *h_factor = s->kind == ROPE_RAMP ? static_cast<float>(0.1 * std::log(s->factor) + 1.0) : 1.f;
  return DEC_OK;
}

extern "C" dec_status qk_norm_rope(const qk_rope_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "qk_norm_rope: NULL arguments");
  dec_status s = check_rows(a, "qk_norm_rope");
  if (s != DEC_OK) return s;
  if (a->rows == 0 || a->n_q + a->n_kv == 0) return DEC_OK;
  if (a->n_kv > 0 && !a->k_out) return fail(nullptr, DEC_EINVAL, "qk_norm_rope: NULL k_out");
  if (a->n_kv > 0 && !aligned_to(elem_bytes(a->ydtype), a->k_out))
    return fail(nullptr, DEC_EINVAL, "qk_norm_rope: k_out is not aligned to its elements");
  if (a->rows > 1 && a->n_kv > 0 && a->k_out_stride < static_cast<long long>(a->n_kv) * a->head_dim)
    return fail(nullptr, DEC_EINVAL, "qk_norm_rope: k_out rows overlap at stride %lld",
                static_cast<long long>(a->k_out_stride));
  if (a->n_q > 0 && !in_place_ok(a->q, a->q_out, a->rows, a->xdtype, a->ydtype, a->q_stride, a->q_out_stride))
    return fail(nullptr, DEC_EINVAL, "qk_norm_rope: q_out over q needs q's type and stride");
  if (a->n_kv > 0 && !in_place_ok(a->k, a->k_out, a->rows, a->xdtype, a->ydtype, a->k_stride, a->k_out_stride))
    return fail(nullptr, DEC_EINVAL, "qk_norm_rope: k_out over k needs k's type and stride");
  DeviceInfo di;
  if ((s = device_info(&di, nullptr)) != DEC_OK) return s;
  QkRowsArgs k = shared_fields(a);
  k.k_out = a->k_out;
  k.ko_stride = a->k_out_stride;
  k.vec_y = k.vec_y && (a->n_kv == 0 || pieces16(a->k_out, a->k_out_stride, a->ydtype));
  k.err = di.err;
  return run_rows(k, a->xdtype, di, static_cast<cudaStream_t>(stream));
}

extern "C" dec_status kv_append_paged(const kv_append_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "kv_append_paged: NULL arguments");
  dec_status s = check_rows(a, "kv_append_paged");
  if (s != DEC_OK) return s;
  if (a->n_kv < 1) return fail(nullptr, DEC_EINVAL, "kv_append_paged: n_kv must be >= 1");
  if (!is_float(a->kvdtype)) return fail(nullptr, DEC_EINVAL, "kv_append_paged: kvdtype %d", a->kvdtype);
  const int shift = page_shift(a->page_size);
  if (shift < 0)
    return fail(nullptr, DEC_EINVAL, "kv_append_paged: page_size must be a power of two up to %d, got %d", kPageSizeMax,
                a->page_size);
  if (a->n_seq < 0 || a->num_pages < 0 || a->table_stride < 0 || a->base_pos < 0 || a->v_stride < 0)
    return fail(nullptr, DEC_EINVAL, "kv_append_paged: n_seq %d, num_pages %d, table_stride %d, base_pos %d", a->n_seq,
                a->num_pages, a->table_stride, a->base_pos);
  if (a->rows == 0) return DEC_OK;
  if (!a->v || !a->k_pages || !a->v_pages || !a->page_table) return fail(nullptr, DEC_EINVAL, "kv_append_paged: NULL pointer");
  if (!aligned16(a->k_pages) || !aligned16(a->v_pages))
    return fail(nullptr, DEC_EINVAL, "kv_append_paged: the pools must be 16-byte aligned");
  if (!aligned_to(elem_bytes(a->xdtype), a->v) || !aligned_to(4, a->page_table, a->seq))
    return fail(nullptr, DEC_EINVAL, "kv_append_paged: a pointer is not aligned to its elements");
  if (a->n_q > 0 && !in_place_ok(a->q, a->q_out, a->rows, a->xdtype, a->ydtype, a->q_stride, a->q_out_stride))
    return fail(nullptr, DEC_EINVAL, "kv_append_paged: q_out over q needs q's type and stride");
  DeviceInfo di;
  if ((s = device_info(&di, nullptr)) != DEC_OK) return s;
  QkRowsArgs k = shared_fields(a);
  k.v = a->v;
  k.v_stride = a->v_stride;
  k.vec_x = k.vec_x && pieces16(a->v, a->v_stride, a->xdtype);
  k.k_out = a->k_pages;
  k.v_out = a->v_pages;
  k.paged = 1;
  k.pool = PagePool{a->num_pages, a->n_kv, shift, a->table_stride};
  k.table = a->page_table;
  k.seq = a->seq;
  k.n_seq = a->n_seq;
  k.base_pos = a->base_pos;
  k.err = di.err;
  k.kv_f32 = a->kvdtype == DEC_F32;
  return run_rows(k, a->xdtype, di, static_cast<cudaStream_t>(stream));
}
