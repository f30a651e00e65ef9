// Partial attention over a float32 cache on warp-level tf32 instructions, and the
// arguments and helpers that the attention kernels for several branches share.
// The partial results join in attn_join_kernel.
//
// An item is up to 16 query rows of one key/value head and a range of its keys:
// rows of all branches over a range of the shared prefix, or the rows of one
// branch over a range of its own pages. A CTA of eight warps takes an item. Each
// warp streams its own blocks of 8 keys with 16-byte asynchronous copies through
// two stages of its own in shared memory, so the main loop has no CTA-wide
// barrier:
//   S = Q K^T (rows x block), masked; running reference maximum and sum of a
//   softmax; P = 2^(S - reference) stays in registers and becomes the A operand of
//   O += P V. The reference moves only when a block's maximum passes it by 2^8, so
//   O is rarely rescaled.
//   At the end the warps' (O, m, l) join through shared memory and the CTA writes
//   one partial result.
//
// Precision: every operand as tf32 value + remainder, three of the four products
// (about 2^-21 relative is lost), float32 sums.
//
// Rows in shared memory are 16 bytes longer than the head, which makes the matrix
// loads of the keys and the scalar loads of the values free of bank conflicts.
// A block's 96 matrix instructions (48 for the scores, 48 for the outputs at head
// size 128) take 192 cycles of the SM, its 8 KB 350 at the SM's share of the
// memory: bound by memory for long ranges of few rows, by latency for short ones,
// where a warp has four blocks in all (tensor pipe 23%, issue 23%, DRAM 23%), by the
// repeated conversions and reads from L2 for many rows (each 16 walk all keys).
// Measured: 16 rows a head x 3,001 keys and 100 own ones a branch 16.8 us a call with
// its join, x 32,768 60 us (4.5 TB/s); 128 rows a head x 8,192 129 us.
#pragma once
#include <cstdint>

#include "attn_plan.h"
#include "common.h"
#include "paging.h"
#include "ptx.cuh"

namespace wsg {

constexpr int kAmThreads = 32 * kAmWarps;
constexpr float kAmMargin = 8.f;  // the reference moves past this margin (log2 units)

struct AmArgs {
  int batch, n_q, n_kv, d, group, rows;  // rows = batch * group
  const void* q;
  long long q_stride;
  const void *pk, *pv;
  int plen;
  long long pstride;
  const void *kp, *vp;
  PagePool pool;
  const int32_t *table, *len;
  // |scale| log2(e), and the scale's sign, which the queries take on: a masked
  // score stays -inf whatever the scale. Scale 0: queries of 0, scale_log2 1.
  float scale_log2;
  int q_sign;
  int q_even;  // two queries at a time can be read
  // Prefix items: item = (split * n_kv + head) * row_groups + row group, a split
  // covering prefix_chunk keys, its slot the split. Behind them the branches' keys:
  // batch * n_kv segments (branch, head) of own_seg blocks of own_block keys in one
  // line, cut into pieces of own_per blocks; piece w of a segment whose first piece
  // is f has the slot own_slot0 + w - f.
  int prefix_items, row_groups, prefix_chunk;
  int own_block, own_slot0;
  long long own_seg, own_per;
  int first;        // the call's first kernel
  float* part_o;    // [slot][batch * n_q][d]
  float2* part_ml;  // [slot][batch * n_q]: (reference, sum)
  uint32_t* err;
};

template <int DP>
struct AmGeom {
  static constexpr int KB = 8;                       // keys a block
  static constexpr int PITCH = DP * 4 + 16;          // bytes a row
  static constexpr int TILE = KB * PITCH;            // keys (or values) of a block
  static constexpr int QBYTES = 2 * (DP / 8) * 32 * 16;
  static constexpr int RING = 2 * 2 * TILE;          // per warp: two stages
  static constexpr int JOIN = kAmWarps * 16 * DP * 4;  // in the place of the rings
  static constexpr int SMEM = QBYTES + (kAmWarps * RING > JOIN ? kAmWarps * RING : JOIN);
};

__device__ __forceinline__ void am_copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void am_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void am_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void am_ld4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void am_ld4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void am_mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void am_mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float am_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x = hi + lo in tf32 (10 mantissa bits each, hi rounded to nearest).
__device__ __forceinline__ void am_split_tf32(float x, uint32_t* hi, uint32_t* lo) {
  const uint32_t h = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  *hi = h;
  *lo = __float_as_uint(x - __uint_as_float(h));
}

// Two floats as PARTS packed bfloat16 pairs (low half: x) that sum to them.
template <int PARTS>
__device__ __forceinline__ void am_split_bf16(float x, float y, uint32_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[i]) : "f"(y), "f"(x));
    x -= __uint_as_float(p[i] << 16);
    y -= __uint_as_float(p[i] & 0xFFFF0000u);
  }
}

// Grid: prefix items, then one CTA per branch, head and piece (own_per 1, a block
// being a whole range of own_block keys).
template <typename QT, int DP>
__global__ void __launch_bounds__(kAmThreads, 1) attn_f32_kernel(const AmArgs a) {
  using G = AmGeom<DP>;
  constexpr int KB = G::KB, NT = DP / 8;
  extern __shared__ __align__(128) unsigned char am_raw[];
  __shared__ float s_m[kAmWarps][16], s_l[kAmWarps][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();  // the join's CTAs may take their places and wait

  // ---- the item ----
  const bool shared_item = static_cast<int>(blockIdx.x) < a.prefix_items;
  int g, row0, nrows, slot, k0, k1, branch = 0;
  if (shared_item) {
    const int rg = blockIdx.x % a.row_groups, t = blockIdx.x / a.row_groups;
    g = t % a.n_kv;
    slot = t / a.n_kv;
    row0 = rg * 16;
    nrows = min(16, a.rows - row0);
    k0 = slot * a.prefix_chunk;
    k1 = min(a.plen, k0 + a.prefix_chunk);
  } else {
    const int t = blockIdx.x - a.prefix_items;
    const int seg = static_cast<int>(t / a.own_seg), split = static_cast<int>(t - seg * a.own_seg);
    g = seg % a.n_kv;
    branch = seg / a.n_kv;
    slot = a.own_slot0 + split;
    row0 = branch * a.group;
    nrows = a.group;
    // (attn_join_kernel reports a longer branch)
    const int n = static_cast<int>(min(static_cast<int64_t>(a.len[branch]), page_capacity(a.pool)));
    k0 = split * a.own_block;
    k1 = min(n, k0 + a.own_block);
    if (k0 >= k1) return;  // attn_join_kernel knows which pieces hold keys
  }
  const int nblk = (k1 - k0 + KB - 1) / KB;
  const int32_t* trow = a.table + static_cast<long long>(branch) * a.pool.width;
  const char* kbase = static_cast<const char*>(shared_item ? a.pk : a.kp);
  const char* vbase = static_cast<const char*>(shared_item ? a.pv : a.vp);

  unsigned char* ring = am_raw + G::QBYTES + warp * G::RING;
  const uint32_t ring32 = smem_u32(ring);
  const int chunks = a.d / 4;  // 16-byte pieces of a key

  // Request block blk into a stage; the mask of its keys that count (those past
  // the range or without a page arrive as zeros).
  constexpr int CP = DP / 4, KPI = 32 / CP > 0 ? 32 / CP : 1;  // 16-byte pieces of a padded row; keys a step
  constexpr int STEPS = KB * CP / 32;
  const int lkey = lane / CP, lc = lane % CP;
  const uint32_t lane_dst = ring32 + lkey * G::PITCH + lc * 16;
  const int row_bytes = a.d * 4;
  const bool whole = shared_item || (1 << a.pool.shift) >= KB;  // a block's keys are contiguous
  auto request = [&](int stage, int blk) -> uint32_t {
    const int k = k0 + blk * KB, n = min(KB, k1 - k);
    const uint32_t dst = lane_dst + stage * 2 * G::TILE;
    if (whole) {
      long long row = a.pstride * g + k;
      bool have = true;
      if (!shared_item) {
        const int page = page_of(a.pool, trow, k);
        have = page >= 0;
        row = have ? pool_row(a.pool, page, g, k) : 0;
        if (!have && lane == 0) atomicOr(a.err, ERR_BAD_PAGE);
      }
      const long long off = row * row_bytes + lkey * row_bytes + lc * 16;
      const char *ks = kbase + off, *vs = vbase + off;
      if (have && n == KB) {
        if (lc < chunks) {
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            am_copy16(dst + i * KPI * G::PITCH, ks + i * (KPI * row_bytes), 16);
            am_copy16(dst + i * KPI * G::PITCH + G::TILE, vs + i * (KPI * row_bytes), 16);
          }
        }
        return 0xffffffffu >> (32 - KB);
      }
      const int lim = have ? n : 0;
      if (lc < chunks) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const bool in = lkey + i * KPI < lim;  // zeros are written where not
          am_copy16(dst + i * KPI * G::PITCH, in ? ks + i * (KPI * row_bytes) : kbase, in ? 16 : 0);
          am_copy16(dst + i * KPI * G::PITCH + G::TILE, in ? vs + i * (KPI * row_bytes) : vbase, in ? 16 : 0);
        }
      }
      return (1u << lim) - 1u;
    }
    // pages shorter than a block: lane `key` looks its own up
    long long row = -1;
    if (lane < n) {
      const int page = page_of(a.pool, trow, k + lane);
      if (page >= 0)
        row = pool_row(a.pool, page, g, k + lane);
      else
        atomicOr(a.err, ERR_BAD_PAGE);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const long long r = __shfl_sync(0xffffffffu, row, lkey + i * KPI);
      if (lc < chunks) {
        const long long off = r < 0 ? 0 : r * row_bytes + lc * 16;
        am_copy16(dst + i * KPI * G::PITCH, kbase + off, r < 0 ? 0 : 16);
        am_copy16(dst + i * KPI * G::PITCH + G::TILE, vbase + off, r < 0 ? 0 : 16);
      }
    }
    return __ballot_sync(0xffffffffu, row >= 0);
  };

  // ---- the first block on its way, then the query rows ----
  uint32_t ok = 0;  // keys of the block in hand that count
  if (warp < nblk) ok = request(0, warp);
  am_commit();
  if (a.d < DP) {  // columns past the head stay zero
    const int pad = DP / 4 - chunks;
    for (int i = lane; i < 2 * 2 * KB * pad; i += 32)
      *reinterpret_cast<uint4*>(ring + (i / pad) * G::PITCH + (chunks + i % pad) * 16) = make_uint4(0, 0, 0, 0);
  }
  for (int i = tid; i < 16 * (DP / 8); i += kAmThreads) {
    // 8 elements of a row, in the order of the A fragments: [part][k step][lane][register]
    const int r = i / (DP / 8), e = i % (DP / 8) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < nrows && e < a.d) {
      const int row = row0 + r;
      const QT* src = static_cast<const QT*>(a.q) + a.q_stride * (row / a.group) +
                      static_cast<long long>(g * a.group + row % a.group) * a.d + e;
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
      uint32_t* f = reinterpret_cast<uint32_t*>(am_raw) + ((e / 8) * 32 + ln) * 4 + reg;
      f[0] = hi;
      f[NT * 32 * 4] = lo;
    }
  }
  __syncthreads();

  // ---- main loop ----
  float o[NT][4] = {};
  float mref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int stage = 0;
  for (int blk = warp; blk < nblk; blk += kAmWarps, stage ^= 1) {
    __syncwarp();  // every lane is done with the block before this one
    const uint32_t next_ok = blk + kAmWarps < nblk ? request(stage ^ 1, blk + kAmWarps) : 0;
    am_commit();
    am_wait<1>();
    __syncwarp();  // this block has landed for every lane
    const uint32_t kt = ring32 + stage * 2 * G::TILE;
    float s[4] = {}, s2[4] = {}, s3[4] = {};  // the remainders' products are chains of their own
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      uint32_t b[4];
      am_ld4(b, kt + (lane & 7) * G::PITCH + kk * 64 + (lane >> 3) * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t bh0, bl0, bh1, bl1;
        am_split_tf32(__uint_as_float(b[2 * h]), &bh0, &bl0);
        am_split_tf32(__uint_as_float(b[2 * h + 1]), &bh1, &bl1);
        const uint4* f = reinterpret_cast<const uint4*>(am_raw) + ((2 * kk + h) * 32 + lane);
        const uint4 fh = f[0], fl = f[NT * 32];
        const uint32_t qh[4] = {fh.x, fh.y, fh.z, fh.w}, ql[4] = {fl.x, fl.y, fl.z, fl.w};
        am_mma8(s, qh, bh0, bh1);
        am_mma8(s2, qh, bl0, bl1);
        am_mma8(s3, ql, bh0, bh1);
      }
    }
    // register j is row lane / 4 + 8 (j / 2), key 2 (lane % 4) + j % 2
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] += s2[j] + s3[j];
      if (!((ok >> (2 * (lane & 3) + (j & 1))) & 1u)) s[j] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(s[2 * h], s[2 * h + 1]);
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * a.scale_log2;
    }
    if (__any_sync(0xffffffffu, mx[0] > mref[0] + kAmMargin || mx[1] > mref[1] + kAmMargin)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nr = mx[h] > mref[h] + kAmMargin ? mx[h] : mref[h];
        const float f = nr == mref[h] ? 1.f : am_exp2(mref[h] - nr);  // 0 on the first move
        mref[h] = nr;
        l[h] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float m = mref[h] == -INFINITY ? 0.f : mref[h];  // nothing seen yet: every term is 0
#pragma unroll
      for (int j = 2 * h; j < 2 * h + 2; ++j) s[j] = am_exp2(fmaf(s[j], a.scale_log2, -m));
      l[h] += s[2 * h] + s[2 * h + 1];  // this thread's keys only
    }
    // A column c is key 2 c, column c + 4 key 2 c + 1: the scores' own registers
    uint32_t ph[4], pl[4];
    am_split_tf32(s[0], &ph[0], &pl[0]);
    am_split_tf32(s[2], &ph[1], &pl[1]);
    am_split_tf32(s[1], &ph[2], &pl[2]);
    am_split_tf32(s[3], &ph[3], &pl[3]);
    const unsigned char* vrow = ring + stage * 2 * G::TILE + G::TILE + 2 * (lane & 3) * G::PITCH + (lane >> 2) * 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t bh0, bl0, bh1, bl1;
      am_split_tf32(*reinterpret_cast<const float*>(vrow + n * 32), &bh0, &bl0);
      am_split_tf32(*reinterpret_cast<const float*>(vrow + G::PITCH + n * 32), &bh1, &bl1);
      am_mma8(o[n], ph, bh0, bh1);
      am_mma8(o[n], ph, bl0, bl1);
      am_mma8(o[n], pl, bh0, bh1);
    }
    ok = next_ok;
  }
  am_wait<0>();

  // ---- join the warps ----
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      s_m[warp][h * 8 + (lane >> 2)] = mref[h];
      s_l[warp][h * 8 + (lane >> 2)] = l[h];
    }
  }
  __syncthreads();  // every warp is past its ring
  float* join = reinterpret_cast<float*>(am_raw + G::QBYTES);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = h * 8 + (lane >> 2);
    if (r >= nrows) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAmWarps; ++w) m = fmaxf(m, s_m[w][r]);
    const float f = m == -INFINITY ? 1.f : am_exp2(mref[h] - m);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float2*>(join + (warp * 16 + r) * DP + n * 8 + 2 * (lane & 3)) =
          make_float2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
  }
  __syncthreads();
  const long long total_rows = static_cast<long long>(a.batch) * a.n_q;
  for (int i = tid; i < nrows * (DP / 4); i += kAmThreads) {
    const int r = i / (DP / 4), e = i % (DP / 4) * 4, row = row0 + r;
    if (e >= a.d) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kAmWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(join + (w * 16 + r) * DP + e);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    const long long at = slot * total_rows + static_cast<long long>(row / a.group) * a.n_q + g * a.group + row % a.group;
    *reinterpret_cast<float4*>(a.part_o + at * a.d + e) = x;
    if (e == 0) {
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kAmWarps; ++w) m = fmaxf(m, s_m[w][r]);
#pragma unroll
      for (int w = 0; w < kAmWarps; ++w) sum += m == -INFINITY ? s_l[w][r] : s_l[w][r] * am_exp2(s_m[w][r] - m);
      a.part_ml[at] = make_float2(m, sum);
    }
  }
}

// Launches attn_f32_kernel for a head size; sets its shared-memory limit on its
// first launch on a device.
template <typename QT, int DP>
cudaError_t am_launch_one(const AmArgs& a, int items, int dev, cudaStream_t st) {
  constexpr size_t smem = AmGeom<DP>::SMEM;
  static bool lifted[64] = {};
  if (!lifted[dev]) {
    const cudaError_t e = allow_smem_shared(attn_f32_kernel<QT, DP>, smem);
    if (e != cudaSuccess) return e;
    lifted[dev] = true;
  }
  return launch_k(attn_f32_kernel<QT, DP>, dim3(items), dim3(kAmThreads), smem, st, true, a);
}

template <typename QT>
cudaError_t am_launch(const AmArgs& a, int items, int dev, cudaStream_t st) {
  if (a.d <= 16) return am_launch_one<QT, 16>(a, items, dev, st);
  if (a.d <= 64) return am_launch_one<QT, 64>(a, items, dev, st);
  return am_launch_one<QT, 128>(a, items, dev, st);
}

// The launches over a cache type for float32 or bfloat16 queries
// (attn_shared_f32.cu, attn_shared_bf16.cu). na: rows of a prefix item, 8 or 16; 0:
// no prefix items, beside attn_prefix_tc_kernel.
cudaError_t launch_attn_f32(const AmArgs& a, bool q_f32, int items, int dev, cudaStream_t st);
cudaError_t launch_attn_bf16(const AmArgs& a, bool q_f32, int na, int items, int dev, cudaStream_t st);

}  // namespace wsg
