// Partial attention over a bfloat16 cache on warp-level matrix instructions, for
// few query rows a key: the shared prefix with up to 16 rows a key/value head at
// a time, and the branches' own pages (a branch's group of query heads). The
// partial results join in attn_join_kernel.
//
// The keys are the M side: S^T = K Q^T (16 keys x 8 rows an instruction), so 8
// rows fill an instruction. Queries stay in registers as the B operand. S^T's
// registers, rounded to bfloat16 pairs and transposed 8 x 8 between the lanes,
// are the B operand P^T of O^T += V^T P^T; V^T is read from shared memory by
// transposing matrix loads. Softmax: a running reference maximum and sum a row;
// the reference moves only when a block's maximum passes it by 2^8, so O is
// rarely rescaled.
//
// Each warp streams blocks of 16 keys with 16-byte asynchronous copies through
// two stages of its own, so the main loop has no CTA-wide barrier:
//   prefix CTAs  the warps take the blocks of one range of the prefix in turn and
//                join through shared memory at its end;
//   own CTAs     the blocks of all branches' own keys form one line of
//                batch * n_kv segments of equal capacity; each warp takes an equal
//                piece of it, across segments, and writes a partial result per
//                segment it touches. Blocks behind a branch's last token are
//                skipped.
//
// Precision: float32 sums. Keys and values enter exactly, a float32 query as
// three bfloat16 parts (24 bits, exact), a probability as two (QP 1: bfloat16
// queries, whose result is rounded to 8 bits; 2^-16 is lost) or three parts.
//
// Rows in shared memory are 16 bytes longer than the head: no matrix load has
// bank conflicts. Bound by memory for long ranges (the instructions of a block
// take 24 x 8 cycles of one SM quarter for 8 rows, its 8 KB 350 of the SM's
// copies), by the latencies of a block's steps for short ones. Measured: 4 rows a
// head, head size 64, 20,000 shared keys 11.9 us; 128 rows of float32 queries x
// 8,192 102 us (the prefix is read from L2 for every 16 rows).
#pragma once
#include "attn_mma.cuh"

namespace wsg {

template <int DP, int NR, int WARPS>
struct ArGeom {
  static constexpr int KB = 16;               // keys a block
  static constexpr int PITCH = DP * 2 + 16;   // bytes a row
  static constexpr int TILE = KB * PITCH;     // keys (or values) of a block
  static constexpr int RING = 2 * 2 * TILE;   // per warp: two stages
  static constexpr int JOIN = NR * DP * 4;    // per warp, in the place of the ring
  static constexpr int PER_WARP = RING > JOIN ? RING : JOIN;
  static constexpr int SMEM = WARPS * PER_WARP;
};

__device__ __forceinline__ uint32_t ar_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The state of NR query rows (8 or 16) against a stream of key blocks. Lane: row
// pair 2 (lane % 4) of each tile of 8 rows, key (or head element) lane / 4.
template <typename QT, int DP, int QP, int NR>
struct ArCore {
  static constexpr int PITCH = DP * 2 + 16, TILE = 16 * PITCH;
  static constexpr int T = NR / 8, KK = DP / 16, PP = QP == 1 ? 2 : 3;
  uint32_t q[QP][KK][T][2];
  float o[KK][T][4];
  float m[T][2], l[T][2];

  // Rows r < nrows; row(r) is the address of row r's head.
  template <typename Row>
  __device__ __forceinline__ void load(const AmArgs& a, int nrows, Row row) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int r = t * 8 + (lane >> 2);
      const bool have = r < nrows;
      const QT* src = static_cast<const QT*>(a.q) + (have ? row(r) : 0) + 2 * (lane & 3);
      const int left = have ? a.d - 2 * (lane & 3) : 0;  // elements of the row from src on
      if constexpr (sizeof(QT) == 2) {
        if (a.q_even) {
#pragma unroll
          for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              q[0][k][t][h] = k * 16 + h * 8 < left ? *reinterpret_cast<const uint32_t*>(src + k * 16 + h * 8) : 0u;
        } else {
#pragma unroll
          for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = k * 16 + h * 8;
              q[0][k][t][h] = e < left ? src[e] | (static_cast<uint32_t>(src[e + 1]) << 16) : 0u;
            }
        }
        if (a.q_sign != 1) {
#pragma unroll
          for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) q[0][k][t][h] = a.q_sign == 0 ? 0u : q[0][k][t][h] ^ 0x80008000u;
        }
      } else {
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = k * 16 + h * 8;
            uint32_t p[QP];
            am_split_bf16<QP>(e < left ? src[e] * a.q_sign : 0.f, e < left ? src[e + 1] * a.q_sign : 0.f, p);
#pragma unroll
            for (int i = 0; i < QP; ++i) q[i][k][t][h] = p[i];
          }
      }
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KK; ++k) o[k][t][0] = o[k][t][1] = o[k][t][2] = o[k][t][3] = 0.f;
    }
  }

  // One block: keys at shared address kt, values at kt + TILE, `ok` its keys that count.
  __device__ __forceinline__ void consume(uint32_t kt, uint32_t ok, float scale) {
    const int lane = threadIdx.x & 31;
    const uint32_t vt = kt + TILE;
    float s[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      uint32_t ka[4];
      am_ld4(ka, kt + (lane & 15) * PITCH + k * 32 + (lane >> 4) * 16);
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < QP; ++i) am_mma16(s[t], ka, q[i][k][t][0], q[i][k][t][1]);
    }
    // s[t][2 h + j]: key lane / 4 + 8 h, row 8 t + 2 (lane % 4) + j
    if (ok != 0xffffu) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((ok >> ((lane >> 2) + 8 * (i >> 1))) & 1u)) s[t][i] = -INFINITY;
    }
    uint32_t p[T][PP][2];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[j] = fmaxf(s[t][j], s[t][2 + j]);
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16)) * scale;
      }
      if (__any_sync(0xffffffffu, mx[0] > m[t][0] + kAmMargin || mx[1] > m[t][1] + kAmMargin)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float nr = mx[j] > m[t][j] + kAmMargin ? mx[j] : m[t][j];
          const float f = nr == m[t][j] ? 1.f : am_exp2(m[t][j] - nr);  // 0 on the first move
          m[t][j] = nr;
          l[t][j] *= f;
#pragma unroll
          for (int k = 0; k < KK; ++k) o[k][t][j] *= f, o[k][t][2 + j] *= f;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float mu = m[t][j] == -INFINITY ? 0.f : m[t][j];  // nothing seen yet: every term is 0
        s[t][j] = am_exp2(fmaf(s[t][j], scale, -mu));
        s[t][2 + j] = am_exp2(fmaf(s[t][2 + j], scale, -mu));
        l[t][j] += s[t][j] + s[t][2 + j];  // this lane's keys only
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[PP];
        am_split_bf16<PP>(s[t][2 * h], s[t][2 * h + 1], w);
#pragma unroll
        for (int i = 0; i < PP; ++i) p[t][i][h] = ar_transpose(w[i]);
      }
    }
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      uint32_t va[4];
      am_ld4t(va, vt + ((lane >> 4) * 8 + (lane & 7)) * PITCH + k * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < PP; ++i) am_mma16(o[k][t], va, p[t][i][0], p[t][i][1]);
    }
  }

  // The rows' sums over the lanes' keys.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 4);
        l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 8);
        l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 16);
      }
  }
};

// A block's keys and values into a stage by one warp: key k of head g on,
// n <= 16 of them. Returns the mask of the keys that count (those past n or
// without a page arrive as zeros).
template <int DP>
struct ArCopy {
  static constexpr int PITCH = DP * 2 + 16, TILE = 16 * PITCH;
  static constexpr int CP = DP / 8, KPI = 32 / CP, STEPS = 16 / KPI;  // pieces a padded row; keys a step; steps
  int row_bytes, chunks;
  uint32_t ring;
  int lkey, lc;

  __device__ __forceinline__ ArCopy(int d, unsigned char* at) {
    const int lane = threadIdx.x & 31;
    row_bytes = d * 2;
    chunks = d / 8;
    ring = smem_u32(at);
    lkey = lane / CP, lc = lane % CP;
    if (d < DP)  // columns past the head stay zero
      for (int i = lane; i < 4 * 16 * (CP - chunks); i += 32)
        *reinterpret_cast<uint4*>(at + i / (CP - chunks) * PITCH + (chunks + i % (CP - chunks)) * 16) = make_uint4(0, 0, 0, 0);
  }

  // `row`: the first key's row in the cache; its n keys are contiguous
  __device__ __forceinline__ uint32_t run(int stage, const void* kb, const void* vb, long long row, int n) const {
    const uint32_t dst = ring + stage * 2 * TILE + lkey * PITCH + lc * 16;
    const long long off = row * row_bytes + lkey * row_bytes + lc * 16;
    const char *ks = static_cast<const char*>(kb) + off, *vs = static_cast<const char*>(vb) + off;
    if (lc < chunks) {
      if (n == 16) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          am_copy16(dst + i * KPI * PITCH, ks + i * (KPI * row_bytes), 16);
          am_copy16(dst + i * KPI * PITCH + TILE, vs + i * (KPI * row_bytes), 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const bool in = lkey + i * KPI < n;  // zeros are written where not
          am_copy16(dst + i * KPI * PITCH, in ? ks + i * (KPI * row_bytes) : kb, in ? 16 : 0);
          am_copy16(dst + i * KPI * PITCH + TILE, in ? vs + i * (KPI * row_bytes) : vb, in ? 16 : 0);
        }
      }
    }
    return (1u << n) - 1u;
  }

  // keys k .. k + n - 1 of a branch's pages; `entry` is the table's for key k
  __device__ __forceinline__ uint32_t pages(const AmArgs& a, int stage, const int32_t* trow, int32_t entry, int g, int k,
                                            int n) const {
    const int lane = threadIdx.x & 31;
    if (a.pool.shift >= 4) {  // the block lies in one page
      const int page = entry >= 0 && entry < a.pool.num_pages ? entry : -1;
      if (page < 0 && lane == 0) atomicOr(a.err, ERR_BAD_PAGE);
      return run(stage, a.kp, a.vp, page < 0 ? 0 : pool_row(a.pool, page, g, k), page < 0 ? 0 : n);
    }
    long long row = -1;  // lane `key` looks its own page up
    if (lane < n) {
      const int page = page_of(a.pool, trow, k + lane);
      if (page >= 0)
        row = pool_row(a.pool, page, g, k + lane);
      else
        atomicOr(a.err, ERR_BAD_PAGE);
    }
    const uint32_t dst = ring + stage * 2 * TILE + lkey * PITCH + lc * 16;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const long long r = __shfl_sync(0xffffffffu, row, lkey + i * KPI);
      if (lc < chunks) {
        const long long off = r < 0 ? 0 : r * row_bytes + lc * 16;
        am_copy16(dst + i * KPI * PITCH, static_cast<const char*>(a.kp) + off, r < 0 ? 0 : 16);
        am_copy16(dst + i * KPI * PITCH + TILE, static_cast<const char*>(a.vp) + off, r < 0 ? 0 : 16);
      }
    }
    return __ballot_sync(0xffffffffu, row >= 0);
  }
};

// Eight more partial results of a row (reference and sum p, elements y) into (m, l,
// x); p = (-inf, 0) and y = 0 is none. A part whose scores are all -inf has the
// sum 0; a NaN in it stays one.
__device__ __forceinline__ void ar_merge8(const float2 (&p)[8], const float4 (&y)[8], float* m, float* l, float4* x) {
  float mn = *m;
#pragma unroll
  for (int i = 0; i < 8; ++i) mn = fmaxf(mn, p[i].x);
  const float mu = mn == -INFINITY ? 0.f : mn, f = am_exp2(*m - mu);
  *l *= f;
  x->x *= f, x->y *= f, x->z *= f, x->w *= f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float e = p[i].x == -INFINITY ? 1.f : am_exp2(p[i].x - mu);
    *l = fmaf(p[i].y, e, *l);
    x->x = fmaf(y[i].x, e, x->x), x->y = fmaf(y[i].y, e, x->y), x->z = fmaf(y[i].z, e, x->z), x->w = fmaf(y[i].w, e, x->w);
  }
  *m = mn;
}

// NA, NB: rows of a prefix item (8 or 16; 0: no prefix items) and of a branch (8,
// or 16 for groups over 8). CTAs below a.prefix_items are prefix items, the others
// own CTAs. Eight warps, one CTA an SM, where the prefix is cut here (few splits to
// join: 4 x 32768 takes 34 us with three CTAs of four warps an SM, 28 with a third
// of the splits); four warps beside attn_prefix_tc_kernel, whose CTAs leave 152
// registers a thread and 90 KB of shared memory for one.
template <typename QT, int DP, int QP, int NA, int NB>
__global__ void __launch_bounds__(NA ? 256 : 128, NA ? 1 : 3) attn_rows_kernel(const AmArgs a) {
  constexpr int WARPS = NA ? 8 : 4;
  using G = ArGeom<DP, NA, WARPS>;
  constexpr int PER_WARP = G::PER_WARP;
  extern __shared__ __align__(128) unsigned char am_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* mine = am_raw + warp * PER_WARP;
  const ArCopy<DP> copy(a.d, mine);
  const uint32_t ring = smem_u32(mine);
  const long long total_rows = static_cast<long long>(a.batch) * a.n_q;
  // The call's first kernel waits for the stream's previous one; as the second
  // it runs beside attn_prefix_tc_kernel, which has waited before it let it start.
  if (a.first) pdl_wait();
  pdl_trigger();  // the join's CTAs may take their places and wait

  if (NA && static_cast<int>(blockIdx.x) < a.prefix_items) {
    if constexpr (NA > 0) {
      __shared__ float s_m[WARPS][NA], s_l[WARPS][NA];
      const int rg = blockIdx.x % a.row_groups, t0 = blockIdx.x / a.row_groups;
      const int g = t0 % a.n_kv, slot = t0 / a.n_kv;
      const int row0 = rg * NA, nrows = min(NA, a.rows - row0);
      const int k0 = slot * a.prefix_chunk, k1 = min(a.plen, k0 + a.prefix_chunk);
      const int nblk = (k1 - k0 + 15) / 16;
      auto request = [&](int stage, int blk) {
        const int k = k0 + blk * 16;
        return copy.run(stage, a.pk, a.pv, a.pstride * g + k, min(16, k1 - k));
      };
      uint32_t ok = 0;
      if (warp < nblk) ok = request(0, warp);
      am_commit();
      auto place = [&](int r) {  // row r of this item among all (branch, query head) rows
        return static_cast<long long>((row0 + r) / a.group) * a.n_q + g * a.group + (row0 + r) % a.group;
      };
      ArCore<QT, DP, QP, NA> core;
      core.load(a, nrows, [&](int r) {
        return a.q_stride * ((row0 + r) / a.group) + static_cast<long long>(g * a.group + (row0 + r) % a.group) * a.d;
      });
      int stage = 0;
      for (int blk = warp; blk < nblk; blk += WARPS, stage ^= 1) {
        __syncwarp();  // every lane is done with the block before this one
        const uint32_t next = blk + WARPS < nblk ? request(stage ^ 1, blk + WARPS) : 0;
        am_commit();
        am_wait<1>();
        __syncwarp();  // this block has landed for every lane
        core.consume(ring + stage * 2 * G::TILE, ok, a.scale_log2);
        ok = next;
      }
      am_wait<0>();
      core.finish();
      // ---- join the warps ----
  #pragma unroll
      for (int t = 0; t < NA / 8; ++t)
  #pragma unroll
        for (int j = 0; j < 2; ++j)
          if (lane < 4) {
            s_m[warp][t * 8 + 2 * lane + j] = core.m[t][j];
            s_l[warp][t * 8 + 2 * lane + j] = core.l[t][j];
          }
      __syncthreads();  // every warp is past its ring
      float* out = reinterpret_cast<float*>(mine);
  #pragma unroll
      for (int t = 0; t < NA / 8; ++t)
  #pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = t * 8 + 2 * (lane & 3) + j;
          if (r >= nrows) continue;
          float m = -INFINITY;
  #pragma unroll
          for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_m[w][r]);
          const float f = m == -INFINITY ? 1.f : am_exp2(core.m[t][j] - m);
  #pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            out[r * DP + k * 16 + (lane >> 2)] = core.o[k][t][j] * f;
            out[r * DP + k * 16 + 8 + (lane >> 2)] = core.o[k][t][2 + j] * f;
          }
        }
      __syncthreads();
      for (int i = tid; i < nrows * (DP / 4); i += 32 * WARPS) {
        const int r = i / (DP / 4), e = i % (DP / 4) * 4;
        if (e >= a.d) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(am_raw + w * PER_WARP + (r * DP + e) * 4);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const long long at = slot * total_rows + place(r);
        *reinterpret_cast<float4*>(a.part_o + at * a.d + e) = x;
        if (e == 0) {
          float m = -INFINITY, sum = 0.f;
  #pragma unroll
          for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_m[w][r]);
  #pragma unroll
          for (int w = 0; w < WARPS; ++w) sum += m == -INFINITY ? s_l[w][r] : s_l[w][r] * am_exp2(s_m[w][r] - m);
          a.part_ml[at] = make_float2(m, sum);
        }
      }
    }
  } else {
    // ---- this warp's piece of the line of own blocks ----
    const long long w = static_cast<long long>(blockIdx.x - a.prefix_items) * WARPS + warp;
    const long long end = min((w + 1) * a.own_per, static_cast<long long>(a.batch) * a.n_kv * a.own_seg);
    // A block of the line: branch, head, first key, keys that count, the table's
    // entry of its page. Positions advance without divisions, and a block's entry
    // is read one block before its keys are requested.
    struct Block {
      int b, g, k, n;
      int32_t entry;
      bool have;
    };
    int left = w * a.own_per < end ? static_cast<int>(end - w * a.own_per) : 0;  // blocks of the piece from `at` on
    int b = 0, g = 0, held = -1;
    long long at = 0;  // block within the segment
    if (left > 0) {
      const long long seg = w * a.own_per / a.own_seg;
      at = w * a.own_per - seg * a.own_seg;
      b = static_cast<int>(seg / a.n_kv);
      g = static_cast<int>(seg % a.n_kv);
    }
    // the next block that holds keys
    auto take = [&]() {
      Block x{};
      while (left > 0) {
        if (at == a.own_seg) {
          at = 0;
          if (++g == a.n_kv) g = 0, ++b, held = -1;
        }
        if (held < 0) {
          // (attn_join_kernel reports a longer branch)
          held = static_cast<int>(min(static_cast<int64_t>(max(0, a.len[b])), page_capacity(a.pool)));
        }
        const int k = static_cast<int>(at) * 16;
        if (k < held) {
          x.b = b, x.g = g, x.k = k, x.n = min(16, held - k), x.have = true;
          if (a.pool.shift >= 4) x.entry = a.table[static_cast<long long>(b) * a.pool.width + (k >> a.pool.shift)];
          ++at;
          --left;
          return x;
        }
        left -= static_cast<int>(min(static_cast<long long>(left), a.own_seg - at));
        at = a.own_seg;
      }
      return x;
    };
    auto request = [&](int stage, const Block& x) {
      return copy.pages(a, stage, a.table + static_cast<long long>(x.b) * a.pool.width, x.entry, x.g, x.k, x.n);
    };
    ArCore<QT, DP, QP, NB> core;
    int lb = -1, lg = 0;  // the branch and head whose rows are in the core
    auto flush = [&]() {
      core.finish();
      const long long slot = a.own_slot0 + w - (static_cast<long long>(lb) * a.n_kv + lg) * a.own_seg / a.own_per;
#pragma unroll
      for (int t = 0; t < NB / 8; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = t * 8 + 2 * (lane & 3) + j;
          if (r >= a.group) continue;
          const long long at = slot * total_rows + static_cast<long long>(lb) * a.n_q + lg * a.group + r;
          float* o = a.part_o + at * a.d + (lane >> 2);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            if (k * 16 < a.d) o[k * 16] = core.o[k][t][j];
            if (k * 16 + 8 < a.d) o[k * 16 + 8] = core.o[k][t][2 + j];
          }
          if (lane < 4) a.part_ml[at] = make_float2(core.m[t][j], core.l[t][j]);
        }
    };
    Block cur = take(), next = take();
    uint32_t ok = 0;
    if (cur.have) ok = request(0, cur);
    am_commit();
    int stage = 0;
    while (cur.have) {
      __syncwarp();  // every lane is done with the block before this one
      const uint32_t next_ok = next.have ? request(stage ^ 1, next) : 0;
      am_commit();
      const Block after = take();
      if (cur.b != lb || cur.g != lg) {
        if (lb >= 0) flush();
        lb = cur.b, lg = cur.g;
        const long long base = a.q_stride * lb + static_cast<long long>(lg) * a.group * a.d;
        core.load(a, a.group, [&](int r) { return base + static_cast<long long>(r) * a.d; });
      }
      am_wait<1>();
      __syncwarp();  // this block has landed for every lane
      core.consume(ring + stage * 2 * G::TILE, ok, a.scale_log2);
      cur = next;
      next = after;
      ok = next_ok;
      stage ^= 1;
    }
    am_wait<0>();
    if (lb >= 0) flush();
  }
  // This launch may run beside attn_prefix_tc_kernel: it ends after that one, so
  // that the join, which waits for this launch, finds both.
  pdl_wait();
}

template <typename QT, int DP, int QP, int NA, int NB>
cudaError_t ar_launch_one(const AmArgs& a, int items, int dev, cudaStream_t st) {
  constexpr int WARPS = NA ? 8 : 4;
  constexpr size_t smem = ArGeom<DP, NA, WARPS>::SMEM;
  static bool lifted[64] = {};
  if (!lifted[dev]) {
    const cudaError_t e = allow_smem_shared(attn_rows_kernel<QT, DP, QP, NA, NB>, smem);
    if (e != cudaSuccess) return e;
    lifted[dev] = true;
  }
  return launch_k(attn_rows_kernel<QT, DP, QP, NA, NB>, dim3(items), dim3(32 * WARPS), smem, st, true, a);
}

template <typename QT, int DP, int QP>
cudaError_t ar_launch_rows(const AmArgs& a, int na, int items, int dev, cudaStream_t st) {
  if (a.group > 8) return ar_launch_one<QT, DP, QP, 16, 16>(a, items, dev, st);
  return na == 16 ? ar_launch_one<QT, DP, QP, 16, 8>(a, items, dev, st)
                  : ar_launch_one<QT, DP, QP, 8, 8>(a, items, dev, st);
}

// na: rows of a prefix item, 8 or 16; 0: own keys only (bfloat16 queries, head size
// 128, whose prefix attn_prefix_tc_kernel takes).
template <typename QT, int QP>
cudaError_t ar_launch(const AmArgs& a, int na, int items, int dev, cudaStream_t st) {
  if constexpr (QP == 1)
    if (na == 0)
      return a.group > 8 ? ar_launch_one<QT, 128, QP, 0, 16>(a, items, dev, st)
                         : ar_launch_one<QT, 128, QP, 0, 8>(a, items, dev, st);
  if (a.d <= 16) return ar_launch_rows<QT, 16, QP>(a, na, items, dev, st);
  if (a.d <= 64) return ar_launch_rows<QT, 64, QP>(a, na, items, dev, st);
  return ar_launch_rows<QT, 128, QP>(a, na, items, dev, st);
}

}  // namespace wsg
