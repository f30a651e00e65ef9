// Attention of a step's rows on warp-level matrix instructions, for every type, head
// size and page size: row tiles of 16, 32 or 64 rows (attn_tree_plan.h), a CTA a share of
// the line of key tiles. Its warps are RG groups of 16 rows times KG rings: the warps of a
// ring stream blocks of keys through it together, each copying a part, and each
// holds its 16 rows against every block (attn_rows.cuh: bfloat16 caches, blocks of 16 keys
// as the M side; float32 caches as in attn_mma.cuh: blocks of 8 keys, tf32 value and
// remainder, three products). So the keys are read once for up to 64 rows.
//
// Bound by a block's chain of instructions for many rows and for float32, by memory for few
// rows of bfloat16. Measured (16 query heads over 8, heads of 128, all requests as long as said): 32
// single tokens x 4,096 bfloat16 98 us (5.5 TB/s), float32 queries 103, float32 caches 214 (5.0
// TB/s; bfloat16 queries over them 180); 32 x 64 rows 693, 1,545 and 1,144.
//
// Blocks that hold drafted rows' keys mask scores row by row. A value that is not
// finite would reach rows that do not see it through its product with a weight of 0,
// so in these blocks it enters the products as 0 and is added afterwards to the rows
// that see it, which it makes not finite.
#pragma once
#include "attn_tree.cuh"

namespace wsg {

__device__ __forceinline__ bool at_odd(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }

// D = A B, the first product of a sum. The matrix instructions cut their sums off where
// an addition would round, always towards 0: over many keys that is a share of the result
// (32 x 64 rows x 16,384 tokens: error 5.7e-5, against 7.8e-7), and bfloat16 results next to a
// border round to its other side. So a block's products are summed from 0 and added by themselves
// (float32 results 5 to 18% of the time, bfloat16 ones over bfloat16 caches 2 to 10%). Bfloat16
// results over float32 caches are summed in the instructions over 64 blocks, 192 instructions that
// lose some 3e-6, and these sums added up in memory: 4% of the time, 15 if every block's were.
__device__ __forceinline__ void at_mma16z(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void at_mma8z(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// x += y, two elements an instruction.
__device__ __forceinline__ void at_add4(float (&x)[4], const float (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %3};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
        : "+f"(x[i]), "+f"(x[i + 1])
        : "f"(y[i]), "f"(y[i + 1]));
}

// ---- bfloat16 caches -------------------------------------------------------------

template <typename QT, int DP, int QP>
struct AtCore16 : ArCore<QT, DP, QP, 16> {
  using Base = ArCore<QT, DP, QP, 16>;
  static constexpr int KB = 16, TILE = Base::TILE, PITCH = Base::PITCH, KK = Base::KK, PP = Base::PP;
  static constexpr bool APART = true;  // a block's products are added by themselves

  // row, keys' words: seen[t][j] of row 8 t + 2 (lane % 4) + j
  __device__ __forceinline__ static int row_of(int i) { return 8 * (i >> 1) + 2 * (threadIdx.x & 3) + (i & 1); }

  // DRAFTS: scores masked by row, and values that are not finite added afterwards. Products
  // into one accumulator stand apart: back to back each would wait for the one before it
  // (two warps a scheduler do not hide that).
  template <bool DRAFTS>
  __device__ __forceinline__ void consume_block(uint32_t kt, const unsigned char* vp, uint32_t ok, float scale,
                                                const uint32_t (&seen)[4]) {
    const int lane = threadIdx.x & 31;
    const uint32_t vt = kt + TILE;
    constexpr int CH = QP == 1 ? 2 : QP;  // chains of sums a row group: k steps by parity, or the queries' parts
    float sc[CH][2][4] = {};
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      uint32_t ka[4];
      am_ld4(ka, kt + (lane & 15) * PITCH + k * 32 + (lane >> 4) * 16);
#pragma unroll
      for (int i = 0; i < QP; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) am_mma16(sc[QP == 1 ? k & 1 : i][t], ka, this->q[i][k][t][0], this->q[i][k][t][1]);
    }
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i] = sc[CH - 1][t][i];
#pragma unroll
        for (int c = CH - 2; c >= 0; --c) s[t][i] += sc[c][t][i];
        const uint32_t may = DRAFTS ? ok & seen[2 * t + (i & 1)] : ok;
        if (!((may >> ((lane >> 2) + 8 * (i >> 1))) & 1u)) s[t][i] = -INFINITY;
      }
    float mx[2][2];
    bool move = false;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) mx[t][j] = fmaxf(s[t][j], s[t][2 + j]);
#pragma unroll
    for (int d = 4; d < 32; d *= 2)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) mx[t][j] = fmaxf(mx[t][j], __shfl_xor_sync(0xffffffffu, mx[t][j], d));
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) mx[t][j] *= scale, move |= mx[t][j] > this->m[t][j] + kAmMargin;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float nr = mx[t][j] > this->m[t][j] + kAmMargin ? mx[t][j] : this->m[t][j];
          const float f = nr == this->m[t][j] ? 1.f : am_exp2(this->m[t][j] - nr);  // 0 on the first move
          this->m[t][j] = nr;
          this->l[t][j] *= f;
#pragma unroll
          for (int k = 0; k < KK; ++k) this->o[k][t][j] *= f, this->o[k][t][2 + j] *= f;
        }
    }
    uint32_t p[2][PP][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float mu = this->m[t][j] == -INFINITY ? 0.f : this->m[t][j];  // nothing seen yet: every term is 0
        s[t][j] = am_exp2(fmaf(s[t][j], scale, -mu));
        s[t][2 + j] = am_exp2(fmaf(s[t][2 + j], scale, -mu));
        this->l[t][j] += s[t][j] + s[t][2 + j];  // this lane's keys only
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[PP];
        am_split_bf16<PP>(s[t][2 * h], s[t][2 * h + 1], w);
#pragma unroll
        for (int i = 0; i < PP; ++i) p[t][i][h] = ar_transpose(w[i]);
      }
    }
    bool odd = false;
    constexpr int KS = KK < 2 || sizeof(QT) == 4 ? 1 : 2;  // k steps at a time
#pragma unroll
    for (int k = 0; k < KK; k += KS) {
      uint32_t va[KS][4];
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        am_ld4t(va[u], vt + ((lane >> 4) * 8 + (lane & 7)) * PITCH + (k + u) * 32 + ((lane >> 3) & 1) * 16);
        if (DRAFTS) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t c = at_finite2(va[u][i]);
            odd |= c != va[u][i];
            va[u][i] = c;
          }
        }
      }
      float c[KS][2][4];
#pragma unroll
      for (int i = PP - 1; i >= 0; --i)
#pragma unroll
        for (int u = 0; u < KS; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (i == PP - 1)
              at_mma16z(c[u][t], va[u], p[t][i][0], p[t][i][1]);
            else
              am_mma16(c[u][t], va[u], p[t][i][0], p[t][i][1]);
          }
#pragma unroll
      for (int u = 0; u < KS; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) at_add4(this->o[k + u][t], c[u][t]);
    }
    if (DRAFTS && __any_sync(0xffffffffu, odd)) {
      for (int key = 0; key < 16; ++key)
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint16_t v = *reinterpret_cast<const uint16_t*>(vp + key * PITCH + (k * 16 + h * 8 + (lane >> 2)) * 2);
            if (!at_odd16(v)) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if ((ok & seen[2 * t + j]) >> key & 1u) this->o[k][t][2 * h + j] += bf16_to_f32(v);
          }
    }
  }

  __device__ __forceinline__ void block(uint32_t kt, const unsigned char* vp, uint32_t ok, float scale, bool drafts,
                                        const uint32_t (&seen)[4]) {
    if (drafts)
      consume_block<true>(kt, vp, ok, scale, seen);
    else
      consume_block<false>(kt, vp, ok, scale, seen);
  }

  // each row's reference and sum, one lane a row
  template <typename F>
  __device__ __forceinline__ void sums(F put) {
    const int lane = threadIdx.x & 31;
    this->finish();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane < 4) put(t * 8 + 2 * lane + j, this->m[t][j], this->l[t][j]);
  }
  // outputs of row r times f(r, reference) to put(r, element, value)
  template <typename F, typename P>
  __device__ __forceinline__ void outputs(int nrows, F f, P put) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = t * 8 + 2 * (lane & 3) + j;
        if (r >= nrows) continue;
        const float x = f(r, this->m[t][j]);
#pragma unroll
        for (int k = 0; k < KK; ++k) {
          put(r, k * 16 + (lane >> 2), this->o[k][t][j] * x);
          put(r, k * 16 + 8 + (lane >> 2), this->o[k][t][2 + j] * x);
        }
      }
  }
};

// ---- float32 caches --------------------------------------------------------------

// The state of 16 rows against a stream of blocks of 8 keys; lane: rows lane / 4 and
// that + 8, keys 2 (lane % 4) and the next of a block's scores.
template <typename QT, int DP, int QP>
struct AtCore32 {
  static constexpr int KB = 8, PITCH = DP * 4 + 16, TILE = KB * PITCH, NT = DP / 8;
  static constexpr bool APART = sizeof(QT) == 4;  // a block's products are added by themselves, or those of some blocks

  float o[NT][4];
  float m[2], l[2];
  const uint4* frag;  // queries in shared memory: [part][k step][lane], split once a piece

  __device__ __forceinline__ static int row_of(int i) { return ((threadIdx.x & 31) >> 2) + 8 * (i & 1); }

  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }

  template <bool DRAFTS>
  __device__ __forceinline__ void consume(uint32_t kt, const unsigned char* vp, uint32_t ok, float scale,
                                          const uint32_t (&seen)[4]) {
    const int lane = threadIdx.x & 31;
    float s[4] = {}, s2[4] = {}, s3[4] = {};  // the remainders' products are chains of their own
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      uint32_t b[4];
      am_ld4(b, kt + (lane & 7) * PITCH + kk * 64 + (lane >> 3) * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t bh0, bl0, bh1, bl1;
        am_split_tf32(__uint_as_float(b[2 * h]), &bh0, &bl0);
        am_split_tf32(__uint_as_float(b[2 * h + 1]), &bh1, &bl1);
        const uint4 fh = frag[(2 * kk + h) * 32 + lane], fl = frag[NT * 32 + (2 * kk + h) * 32 + lane];
        const uint32_t qh[4] = {fh.x, fh.y, fh.z, fh.w}, ql[4] = {fl.x, fl.y, fl.z, fl.w};
        am_mma8(s, qh, bh0, bh1);
        am_mma8(s2, qh, bl0, bl1);
        if (sizeof(QT) == 4) am_mma8(s3, ql, bh0, bh1);  // bfloat16 queries have no remainder
      }
    }
    // register j is row lane / 4 + 8 (j / 2), key 2 (lane % 4) + j % 2
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] += s2[j] + s3[j];
      const uint32_t may = DRAFTS ? ok & seen[j >> 1] : ok;
      if (!(may >> (2 * (lane & 3) + (j & 1)) & 1u)) s[j] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(s[2 * h], s[2 * h + 1]);
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * scale;
    }
    if (__any_sync(0xffffffffu, mx[0] > m[0] + kAmMargin || mx[1] > m[1] + kAmMargin)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nr = mx[h] > m[h] + kAmMargin ? mx[h] : m[h];
        const float f = nr == m[h] ? 1.f : am_exp2(m[h] - nr);  // 0 on the first move
        m[h] = nr;
        l[h] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mu = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: every term is 0
#pragma unroll
      for (int j = 2 * h; j < 2 * h + 2; ++j) s[j] = am_exp2(fmaf(s[j], scale, -mu));
      l[h] += s[2 * h] + s[2 * h + 1];  // this lane's keys only
    }
    // A column c is key 2 c, column c + 4 key 2 c + 1: the scores' own registers
    uint32_t ph[4], pl[4];
    am_split_tf32(s[0], &ph[0], &pl[0]);
    am_split_tf32(s[2], &ph[1], &pl[1]);
    am_split_tf32(s[1], &ph[2], &pl[2]);
    am_split_tf32(s[3], &ph[3], &pl[3]);
    const unsigned char* vrow = vp + 2 * (lane & 3) * PITCH + (lane >> 2) * 4;
    bool odd = false;
    constexpr int NS = APART || NT < 4 ? 2 : 4;  // columns at a time: products into one accumulator stand apart
#pragma unroll
    for (int n = 0; n < NT; n += NS) {
      float c[NS][4];
      uint32_t bh[NS][2], bl[NS][2];
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = *reinterpret_cast<const float*>(vrow + e * PITCH + (n + u) * 32);
          if (DRAFTS && at_odd(v)) v = 0.f, odd = true;
          am_split_tf32(v, &bh[u][e], &bl[u][e]);
        }
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        if constexpr (APART)
          at_mma8z(c[u], pl, bh[u][0], bh[u][1]);
        else
          am_mma8(o[n + u], pl, bh[u][0], bh[u][1]);
      }
#pragma unroll
      for (int u = 0; u < NS; ++u) am_mma8(APART ? c[u] : o[n + u], ph, bl[u][0], bl[u][1]);
#pragma unroll
      for (int u = 0; u < NS; ++u) am_mma8(APART ? c[u] : o[n + u], ph, bh[u][0], bh[u][1]);
      if constexpr (APART) {
#pragma unroll
        for (int u = 0; u < NS; ++u) at_add4(o[n + u], c[u]);
      }
    }
    if (DRAFTS && __any_sync(0xffffffffu, odd)) {
      for (int key = 0; key < 8; ++key)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float v = *reinterpret_cast<const float*>(vp + key * PITCH + (n * 8 + 2 * (lane & 3) + e) * 4);
            if (!at_odd(v)) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if ((ok & seen[h]) >> key & 1u) o[n][2 * h + e] += v;
          }
    }
  }

  __device__ __forceinline__ void block(uint32_t kt, const unsigned char* vp, uint32_t ok, float scale, bool drafts,
                                        const uint32_t (&seen)[4]) {
    if (drafts)
      consume<true>(kt, vp, ok, scale, seen);
    else
      consume<false>(kt, vp, ok, scale, seen);
  }

  // The sums over earlier blocks lie in `sum`, a row's part and its reference. JOIN: o becomes the
  // whole; otherwise the total takes o in (first: becomes it).
  template <bool JOIN>
  __device__ __forceinline__ void total(volatile float* sum, bool first) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      volatile float* t = sum + h * (2 * NT + 1);
      if (!first) {
        const float ref = t[2 * NT], f = ref == m[h] ? 1.f : am_exp2(ref - m[h]);
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) o[i >> 1][2 * h + (i & 1)] = fmaf(t[i], f, o[i >> 1][2 * h + (i & 1)]);
      }
      if (JOIN) continue;
      t[2 * NT] = m[h];
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) t[i] = o[i >> 1][2 * h + (i & 1)], o[i >> 1][2 * h + (i & 1)] = 0.f;
    }
  }

  template <typename F>
  __device__ __forceinline__ void sums(F put) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if ((lane & 3) == 0) put(h * 8 + (lane >> 2), m[h], l[h]);
    }
  }
  template <typename F, typename P>
  __device__ __forceinline__ void outputs(int nrows, F f, P put) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * 8 + (lane >> 2);
      if (r >= nrows) continue;
      const float x = f(r, m[h]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        put(r, n * 8 + 2 * (lane & 3), o[n][2 * h] * x);
        put(r, n * 8 + 2 * (lane & 3) + 1, o[n][2 * h + 1] * x);
      }
    }
  }
};

// A block's keys and values into a ring slot by the RG warps that share the ring, `part`
// being one of them: each copies every RG-th step. The mask of the keys that count; the
// others arrive as zeros.
template <int KEYS, int ELEM, int DP, int RG>
struct AtCopy {
  static constexpr int PITCH = DP * ELEM + 16, TILE = KEYS * PITCH;
  static constexpr int CP = DP * ELEM / 16, KPI = 32 / CP, STEPS = KEYS / KPI;  // pieces a padded row; keys a step; steps
  static_assert(KPI >= 1 && STEPS >= 1, "a step is a warp's copies");
  int row_bytes, chunks, part, lkey, lc;
  uint32_t ring;

  __device__ __forceinline__ AtCopy(int d, uint32_t ring_, int part_) {
    const int lane = threadIdx.x & 31;
    row_bytes = d * ELEM;
    chunks = row_bytes / 16;
    part = part_;
    ring = ring_;
    lkey = lane / CP, lc = lane % CP;
  }
  __device__ __forceinline__ uint32_t run(int slot, const void* kb, const void* vb, long long row, int n) const {
    const uint32_t dst = ring + slot * 2 * TILE + lkey * PITCH + lc * 16;
    const long long off = row * row_bytes + lkey * row_bytes + lc * 16;
    const char *ks = static_cast<const char*>(kb) + off, *vs = static_cast<const char*>(vb) + off;
    if (lc < chunks) {
#pragma unroll
      for (int j = 0; j < (STEPS + RG - 1) / RG; ++j) {
        const int i = j * RG + part;
        if (STEPS % RG && i >= STEPS) break;
        const bool in = lkey + i * KPI < n;
        am_copy16(dst + i * KPI * PITCH, in ? ks + i * (KPI * row_bytes) : kb, in ? 16 : 0);
        am_copy16(dst + i * KPI * PITCH + TILE, in ? vs + i * (KPI * row_bytes) : vb, in ? 16 : 0);
      }
    }
    return (1u << n) - 1u;
  }
  // keys k .. k + n - 1 of a request's pages; `entry` is the table's for key k
  __device__ __forceinline__ uint32_t pages(const AmArgs& a, int slot, const int32_t* trow, int32_t entry, int g, int k,
                                            int n) const {
    const int lane = threadIdx.x & 31;
    if (1 << a.pool.shift >= KEYS) {  // the block lies in one page
      const int page = entry >= 0 && entry < a.pool.num_pages ? entry : -1;
      if (page < 0 && lane == 0) atomicOr(a.err, ERR_BAD_PAGE);
      return run(slot, a.kp, a.vp, page < 0 ? 0 : pool_row(a.pool, page, g, k), page < 0 ? 0 : n);
    }
    long long row = -1;  // lane `key` looks its own page up
    if (lane < n) {
      const int page = page_of(a.pool, trow, k + lane);
      if (page >= 0)
        row = pool_row(a.pool, page, g, k + lane);
      else
        atomicOr(a.err, ERR_BAD_PAGE);
    }
    const uint32_t dst = ring + slot * 2 * TILE + lkey * PITCH + lc * 16;
#pragma unroll
    for (int j = 0; j < (STEPS + RG - 1) / RG; ++j) {
      const int i = j * RG + part;
      if (STEPS % RG && i >= STEPS) break;
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

// ---- the kernel --------------------------------------------------------------------

// RG groups of 16 rows, KG = WARPS / RG rings of blocks; SLOTS blocks of a ring. The work on
// a float32 block is one long chain (tensor pipe and issue slots 28 and 26% busy with 8 warps):
// 12 warps, two blocks each, take 214 us for 32 rows x 4,096, 8 warps 245. For bfloat16 the
// queries' parts leave no registers for more; they run as PER CTAs of 8 / PER warps an SM, so
// that segments of few keys do not wait for each other's chains (attn_tree_plan.h).
template <typename QT, int DP, bool F32, int RG, int PER>
struct AtGeom {
  static constexpr int WARPS = F32 ? 12 : 8 / PER, KG = WARPS / RG;
  static constexpr int BLOCK = F32 ? 2 * 8 * (DP * 4 + 16) : 2 * 16 * (DP * 2 + 16);
  static constexpr int SLOTS = F32 ? (RG == 1 ? 2 : 6) : RG == 1 ? 3 : RG == 2 ? 5 : 8;
  static constexpr int RING = SLOTS * BLOCK;
  static constexpr int JOIN = WARPS * 16 * DP * 4;
  static constexpr int QBYTES = F32 ? RG * 2 * (DP / 8) * 32 * 16 : 0;
  static constexpr int SMEM = QBYTES + (KG * RING > JOIN ? KG * RING : JOIN);
};

template <typename QT, int DP, int QP, bool F32, int RG, int PER>
__global__ void __launch_bounds__(32 * AtGeom<QT, DP, F32, RG, PER>::WARPS, PER) attn_tree_rows_kernel(const AtArgs p) {
  using G = AtGeom<QT, DP, F32, RG, PER>;
  using Core = std::conditional_t<F32, AtCore32<QT, DP, QP>, AtCore16<QT, DP, QP>>;
  constexpr int WARPS = G::WARPS, KG = G::KG, KB = Core::KB, NTHREADS = 32 * WARPS, SLOTS = G::SLOTS;
  extern __shared__ __align__(128) unsigned char am_raw[];
  __shared__ AtWalk s_walk;
  __shared__ AtPiece s_piece;
  __shared__ float s_m[WARPS][16], s_l[WARPS][16];
  const AmArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = warp % RG, kg = warp / RG;  // this warp's rows and ring
  unsigned char* ring = am_raw + G::QBYTES + kg * G::RING;
  const uint32_t ring32 = smem_u32(ring);
  const AtCopy<KB, F32 ? 4 : 2, DP, RG> copy(a.d, ring32, rg);
  // the warps that share a ring
  auto meet = [&]() {
    if constexpr (RG == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * RG) : "memory");
  };
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    AtWalk w = at_start(p);
    const AtPiece x = w.next(p);
    if (lane == 0) s_walk = w, s_piece = x;
  }
  if (warp == 1 && p.prefix_tiles > 0) at_records(p);
  __syncthreads();
  while (s_piece.tiles > 0) {
    const AtPiece pc = s_piece;
    if (a.d < DP) {  // columns past the head stay zero
      constexpr int CP = DP * (F32 ? 4 : 2) / 16;
      const int chunks = a.d * (F32 ? 4 : 2) / 16, pad = CP - chunks;
      for (int i = lane + 32 * rg; i < SLOTS * 2 * KB * pad; i += 32 * RG)
        *reinterpret_cast<uint4*>(ring + i / pad * Core::PITCH + (chunks + i % pad) * 16) = make_uint4(0, 0, 0, 0);
    }
    const int row0 = pc.m0 + 16 * rg, nrows = min(16, pc.nrows - 16 * rg);  // this warp's (none: below 1)
    auto src_of = [&](int r) {
      const int m = row0 + r, token = m / a.group;
      return a.q_stride * (pc.begin + token) + static_cast<long long>(pc.g * a.group + m - token * a.group) * a.d;
    };
    const int32_t* trow = pc.prefix ? nullptr : a.table + static_cast<long long>(pc.s) * a.pool.width;
    const int nblk = max(0, (pc.k1 - pc.k0 + KB - 1) / KB);
    auto entry = [&](int blk) {
      return !pc.prefix && blk < nblk && (KB >> a.pool.shift) <= 1 ? trow[(pc.k0 + blk * KB) >> a.pool.shift] : 0;
    };
    // block number kg + KG i of the piece to slot i
    int32_t e_next = entry(kg);
    auto request = [&](int i) -> uint32_t {
      const int blk = kg + KG * i, slot = i % SLOTS;
      uint32_t ok = 0;
      if (blk < nblk) {
        const int k = pc.k0 + blk * KB, n = min(KB, pc.k1 - k);
        ok = pc.prefix ? copy.run(slot, a.pk, a.pv, a.pstride * pc.g + k, n) : copy.pages(a, slot, trow, e_next, pc.g, k, n);
        e_next = entry(blk + KG);
      }
      am_commit();
      return ok;
    };
    uint32_t ok[SLOTS];  // of the blocks on their way: keys that count (the oldest first)
    ok[SLOTS - 1] = 0;
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) ok[i] = request(i);
    Core core;
    if constexpr (F32) {
      core.clear();
      core.frag = reinterpret_cast<const uint4*>(am_raw) + rg * 2 * (DP / 8) * 32;
      for (int i = tid; i < 16 * RG * (DP / 8); i += NTHREADS) {
        // 8 elements of a row, in the order of the A fragments: [row group][part][k step][lane][register]
        const int rr = i / (DP / 8), e = i % (DP / 8) * 8, r = rr & 15;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (rr < pc.nrows && e < a.d) {
          const int m = pc.m0 + rr, token = m / a.group;
          const QT* src = static_cast<const QT*>(a.q) + a.q_stride * (pc.begin + token) +
                          static_cast<long long>(pc.g * a.group + m - token * a.group) * a.d + e;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(QT) == 4)
              x[j] = src[j] * a.q_sign;
            else
              x[j] = bf16_to_f32(src[j]) * a.q_sign;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ln = (r % 8) * 4 + j % 4, reg = r / 8 + 2 * (j / 4);
          uint32_t hi, lo;
          am_split_tf32(x[j], &hi, &lo);
          uint32_t* f = reinterpret_cast<uint32_t*>(am_raw) + (rr >> 4) * 2 * (DP / 8) * 32 * 4 + ((e / 8) * 32 + ln) * 4 + reg;
          f[0] = hi;
          f[(DP / 8) * 32 * 4] = lo;
        }
      }
      __syncthreads();
    } else {
      core.load(a, nrows, src_of);
    }
    int token[4];  // of the rows whose scores this lane masks
#pragma unroll
    for (int i = 0; i < 4; ++i) token[i] = min(row0 + Core::row_of(i), pc.m0 + pc.nrows - 1) / a.group;
    const int mine = (nblk - kg + KG - 1) / KG;  // blocks of this ring
    constexpr int SUM = Core::APART ? 0 : 64;    // blocks whose products the matrix instructions sum; 0: one
    volatile float total[SUM ? DP / 2 + 4 : 1];  // (in memory)
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      am_wait<SLOTS - 2>();
      meet();  // block i has landed for every warp of the ring, and all are done with the block before it
      ok[SLOTS - 1] = request(i + SLOTS - 1);
      if (nrows > 0) {
        const int k = pc.k0 + (kg + KG * i) * KB;
        const bool drafts = !pc.prefix && k + KB > pc.n;
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        if (drafts)
#pragma unroll
          for (int j = 0; j < 4; ++j) seen[j] = at_seen(p, pc.begin, token[j], k - pc.n);
        const int at = i % SLOTS * 2 * Core::TILE;
        core.block(ring32 + at, ring + at + Core::TILE, ok[0], a.scale_log2, drafts, seen);
      }
      if constexpr (SUM > 0)
        if (i % SUM == SUM - 1 && i + 1 < mine) core.template total<false>(total, i == SUM - 1);
#pragma unroll
      for (int j = 0; j < SLOTS - 1; ++j) ok[j] = ok[j + 1];
    }
    am_wait<0>();
    if constexpr (SUM > 0)
      if (mine > SUM) core.template total<true>(total, false);
    core.sums([&](int r, float m, float l) { s_m[warp][r] = m, s_l[warp][r] = l; });
    __syncthreads();  // every warp is past its ring
    float* out = reinterpret_cast<float*>(am_raw + G::QBYTES) + warp * 16 * DP;
    core.outputs(
        nrows,
        [&](int r, float mine_m) {
          float m = -INFINITY;
#pragma unroll
          for (int w = 0; w < KG; ++w) m = fmaxf(m, s_m[w * RG + rg][r]);
          return m == -INFINITY ? 1.f : am_exp2(mine_m - m);
        },
        [&](int r, int e, float x) { out[r * DP + e] = x; });
    // the next piece, while the results are joined
    if (warp == 0) {
      AtWalk w = s_walk;
      const AtPiece x = w.next(p);
      __syncwarp();
      if (lane == 0) s_walk = w, s_piece = x;
    }
    __syncthreads();
    for (int i = tid; i < pc.nrows * (DP / 4); i += NTHREADS) {
      const int row = i / (DP / 4), e = i % (DP / 4) * 4, g16 = row >> 4, r = row & 15;
      if (e >= a.d) continue;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < KG; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(am_raw + G::QBYTES + (((w * RG + g16) * 16 + r) * DP + e) * 4);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        m = fmaxf(m, s_m[w * RG + g16][r]);
      }
#pragma unroll
      for (int w = 0; w < KG; ++w) {
        const float l = s_l[w * RG + g16][r];
        sum += m == -INFINITY ? l : l * am_exp2(s_m[w * RG + g16][r] - m);
      }
      if (pc.whole) {
        const int mrow = pc.m0 + row, tok = mrow / a.group;
        at_put<QT>(p, pc.begin + tok, pc.g * a.group + mrow - tok * a.group, e, x, m, sum);
      } else {
        const long long at = (pc.id << p.cut.mshift) + row;
        *reinterpret_cast<float4*>(a.part_o + at * a.d + e) = x;
        if (e == 0) a.part_ml[at] = make_float2(m, sum);
      }
    }
    __syncthreads();  // the results have left shared memory
  }
  if (warp == 0 && p.prefix_tiles == 0) at_seams(p, s_walk);
}

template <typename QT, int DP, int QP, bool F32, int RG, int PER = 1>
cudaError_t at_launch_one(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  constexpr size_t smem = AtGeom<QT, DP, F32, RG, PER>::SMEM;
  static bool lifted[64] = {};
  if (!lifted[di.device]) {
    const cudaError_t e = allow_smem_shared(attn_tree_rows_kernel<QT, DP, QP, F32, RG, PER>, smem);
    if (e != cudaSuccess) return e;
    lifted[di.device] = true;
  }
  return launch_k(attn_tree_rows_kernel<QT, DP, QP, F32, RG, PER>, dim3(di.sms * PER), dim3(32 * AtGeom<QT, DP, F32, RG, PER>::WARPS), smem, st, true, a);
}

template <typename QT, int DP, int QP, bool F32>
cudaError_t at_launch_rows(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  if constexpr (!F32) {
    if (a.per_sm == 4) return at_launch_one<QT, DP, QP, F32, 1, 4>(a, di, st);
    if (a.per_sm == 2)
      return a.cut.mshift == 4   ? at_launch_one<QT, DP, QP, F32, 1, 2>(a, di, st)
             : a.cut.mshift == 5 ? at_launch_one<QT, DP, QP, F32, 2, 2>(a, di, st)
                                 : at_launch_one<QT, DP, QP, F32, 4, 2>(a, di, st);
    if (a.cut.mshift == 5) return at_launch_one<QT, DP, QP, F32, 2>(a, di, st);
  }
  return a.cut.mshift == 4 ? at_launch_one<QT, DP, QP, F32, 1>(a, di, st) : at_launch_one<QT, DP, QP, F32, 4>(a, di, st);
}

// (heads above 64 are a translation unit of their own)
template <typename QT, int QP, bool F32>
cudaError_t at_launch(const AtArgs& a, const DeviceInfo& di, cudaStream_t st) {
  if (a.a.d <= 16) return at_launch_rows<QT, 16, QP, F32>(a, di, st);
  return at_launch_rows<QT, 64, QP, F32>(a, di, st);
}

}  // namespace wsg
