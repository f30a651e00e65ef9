// Partial attention of up to 128 query rows over a range of the shared prefix on
// the 5th-generation tensor cores: bfloat16 queries, keys and values, head size
// 128. One CTA per (key/value head, block of 128 rows, split of the prefix).
//
// A row of the matrix products is a (branch, query head) of the key/value head,
// one per tensor-memory lane. The pipeline is that of the prompt's attention
// (prefill_attn_tc.cuh), with 128-key tiles:
//   warp 0      one thread streams keys and values (two 128 x 64 boxes a tile,
//               128-byte swizzle) into two-stage rings; the tensor maps end at the
//               prefix's last row, so rows behind it arrive as zeros;
//   warp 1      one thread issues S_j = Q K_j^T one tile ahead, then O += P_j V_j
//               with P_j over the scores in tensor memory;
//   warps 2-9   two threads a row, half of the tile's keys each: masked, scaled
//               scores, reference maximum (moved only past a margin of 2^8, then
//               O is rescaled in place), probabilities as bfloat16 value +
//               remainder, running sums. Warps whose 32 lanes hold no row sit out.
// The result (O, reference, sum) joins the other splits' in attn_join_kernel.
//
// Tensor memory (512 columns): scores / probabilities at 0 and 128, O at 256, Q
// at 384. The products of a tile take 24 x 64 cycles for any number of rows, its
// 64 KB at the SM's share of the measured bandwidth 2,700 at 1.85 GHz: bound by
// memory for one block of rows. Measured with 128 rows and 8 heads: 32,768 keys
// 33 us a call with its join (4.1 TB/s, 4 us of them the first tile's way),
// each further 32,768 20 us (6.6 TB/s). Three stages instead of two are no faster
// and leave no room for a CTA of the branches' own keys beside this one.
//
// Every wait is bounded; on a timeout the CTA records ERR_TC_TIMEOUT, stops,
// waits for its issued MMAs and copies and frees its tensor memory.
#pragma once
#include "attn_mma.cuh"
#include "tc_attn_util.cuh"

namespace wsg {

constexpr int kApStages = 2, kApThreads = 32 * 10;
constexpr uint32_t kApTile = kApKeys * kApD * 2, kApBox = kApTile / 2;
constexpr uint32_t kApTmO = 256, kApTmQ = 384;
constexpr size_t kApSmem = 2 * kApStages * kApTile + 1024;
constexpr int kApPitch = kApD + 4;  // floats a row of O in shared memory
static_assert(kApRows * kApPitch * 4 <= 2 * kApStages * kApTile, "O fits in the rings");

struct ApArgs {
  const uint16_t* q;
  long long q_stride;
  int batch, n_q, n_kv, group, rows;
  int row_blocks, plen, chunk;  // chunk: keys a split covers, a multiple of 128
  float scale_log2;  // as in AmArgs
  int q_sign;
  float* part_o;  // as in AmArgs, the splits in slots 0 ..
  float2* part_ml;
  uint32_t* err;
};

// Grid: blockIdx.x = (split * n_kv + head) * row_blocks + row block. kmap, vmap:
// the prefix as [n_kv][plen][128] in 128-row x 64-column boxes.
__global__ void __maxnreg__(120)
    attn_prefix_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const ApArgs a) {
  extern __shared__ __align__(1024) unsigned char ap_raw[];
  unsigned char* Ks = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(ap_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* Vs = Ks + kApStages * kApTile;
  __shared__ __align__(8) uint64_t k_full[kApStages], k_empty[kApStages], v_full[kApStages], v_empty[kApStages];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_done[2], drain, pair_bar[4];
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail;
  __shared__ float xch[2][2][kApRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rb = blockIdx.x % a.row_blocks, t0 = blockIdx.x / a.row_blocks;
  const int g = t0 % a.n_kv, split = t0 / a.n_kv;
  const int row0 = rb * kApRows, nrows = min(kApRows, a.rows - row0);
  const int k0 = split * a.chunk, k1 = min(a.plen, k0 + a.chunk);
  const int T = (k1 - k0 + kApKeys - 1) / kApKeys;  // >= 1
  const int live = (nrows + 31) / 32;               // lane quarters that hold rows
  volatile int* vfail = &s_fail;

  if (tid == 0) {
    for (int s = 0; s < kApStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 2 * live);
      mbar_init(&o_done[b], 1);
    }
    mbar_init(&drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&pair_bar[i], 64);
    s_fail = 0;
    fence_mbar_init();
    pdl_wait();  // keys and values may come from the previous kernel
    // the first tiles, ahead of everything else in the CTA
    for (int j = 0; j < kApStages && j < T; ++j) {
      unsigned char *kd = Ks + j * kApTile, *vd = Vs + j * kApTile;
      const int y = k0 + j * kApKeys;
      mbar_arrive_expect_tx(&k_full[j], kApTile);
      tma_load_3d_map(kd, &kmap, 0, y, g, &k_full[j]);
      tma_load_3d_map(kd + kApBox, &kmap, 64, y, g, &k_full[j]);
      mbar_arrive_expect_tx(&v_full[j], kApTile);
      tma_load_3d_map(vd, &vmap, 0, y, g, &v_full[j]);
      tma_load_3d_map(vd + kApBox, &vmap, 64, y, g, &v_full[j]);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const int q = warp & 3, half = (warp - 2) >> 2;  // softmax warps: lane quarter, half of the keys / of D
  const int v = q * 32 + lane;
  const bool have = v < nrows;
  const bool works = warp >= 2 && q < live;
  const long long prow = static_cast<long long>((row0 + v) / a.group) * a.n_q + g * a.group + (row0 + v) % a.group;
  pdl_wait();
  pdl_trigger();  // after the wait: the kernel that runs beside this one does not wait itself
  uint32_t qr[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) qr[i] = 0;
  if (works && have) {  // this thread's half of the row: 64 bfloat16 (any alignment of 2 bytes)
    const uint16_t* src = a.q + a.q_stride * ((row0 + v) / a.group) + (g * a.group + (row0 + v) % a.group) * kApD + half * 64;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 w = reinterpret_cast<const uint4*>(src)[i];
        qr[4 * i] = w.x, qr[4 * i + 1] = w.y, qr[4 * i + 2] = w.z, qr[4 * i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) qr[i] = src[2 * i] | (static_cast<uint32_t>(src[2 * i + 1]) << 16);
    }
  }
  if (a.q_sign != 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) qr[i] = a.q_sign == 0 ? 0u : qr[i] ^ 0x80008000u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);  // this warp's lanes
  if (works) {
    tc_st32(tl + kApTmQ + half * 32, qr);
    tc_wait_st();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  auto fail = [&]() {
    *vfail = 1;
    atomicOr(a.err, ERR_TC_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0) {
      int nk = min(kApStages, T), nv = nk;  // tiles requested
      for (int j = kApStages; j < T && !*vfail; ++j) {
        const int s = j % kApStages, y = k0 + j * kApKeys;
        if (!mbar_wait(&k_empty[s], ((j / kApStages) - 1) & 1)) {
          fail();
          break;
        }
        unsigned char *kd = Ks + s * kApTile, *vd = Vs + s * kApTile;
        mbar_arrive_expect_tx(&k_full[s], kApTile);
        tma_load_3d_map(kd, &kmap, 0, y, g, &k_full[s]);
        tma_load_3d_map(kd + kApBox, &kmap, 64, y, g, &k_full[s]);
        nk = j + 1;
        if (!mbar_wait(&v_empty[s], ((j / kApStages) - 1) & 1)) {
          fail();
          break;
        }
        mbar_arrive_expect_tx(&v_full[s], kApTile);
        tma_load_3d_map(vd, &vmap, 0, y, g, &v_full[s]);
        tma_load_3d_map(vd + kApBox, &vmap, 64, y, g, &v_full[s]);
        nv = j + 1;
      }
      // the last copies into each stage have landed before the CTA may end, after a failure too
      for (int s = 0; s < kApStages; ++s) {
        if (s < nk && !mbar_wait(&k_full[s], ((nk - 1 - s) / kApStages) & 1)) fail();
        if (s < nv && !mbar_wait(&v_full[s], ((nv - 1 - s) / kApStages) & 1)) fail();
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idS = tc_idesc(kApRows, kApKeys);
      constexpr uint32_t idO = tc_idesc(kApRows, kApD) | (1u << 16);  // B (values) MN-major
      auto issue_s = [&](int j) -> bool {
        const int s = j % kApStages;
        if (!mbar_wait(&k_full[s], (j / kApStages) & 1)) return false;
        tc_fence_after();
        const uint32_t kb = smem_u32(Ks + s * kApTile), d = tmem + static_cast<uint32_t>((j & 1) * 128);
#pragma unroll
        for (int kk = 0; kk < kApD / 16; ++kk)
          tc_mma_f16_ts(d, tmem + kApTmQ + kk * 8, tc_desc_sw128(kb + (kk >> 2) * kApBox + (kk & 3) * 32), idS, kk != 0);
        tc_commit(&k_empty[s]);
        tc_commit(&s_full[j & 1]);
        return true;
      };
      bool ok = issue_s(0);
      for (int j = 0; ok && j < T; ++j) {
        // S_{j+1} replaces P_{j-1}: it is issued after P_{j-1} V_{j-1} and runs after it
        if (j + 1 < T && !issue_s(j + 1)) {
          ok = false;
          break;
        }
        const int s = j % kApStages;
        if (!mbar_wait(&p_full[j & 1], (j >> 1) & 1) || !mbar_wait(&v_full[s], (j / kApStages) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t vb = smem_u32(Vs + s * kApTile), pb = tmem + static_cast<uint32_t>((j & 1) * 128);
#pragma unroll
        for (int kk = 0; kk < kApKeys / 16; ++kk) {
          const uint64_t db = tc_desc_sw128_mn(vb + kk * 2048, kApBox, 1024);
#pragma unroll
          for (int part = 0; part < 2; ++part)
            tc_mma_f16_ts(tmem + kApTmO, pb + part * 64 + kk * 8, db, idO, (j | kk | part) != 0);
        }
        tc_commit(&v_empty[s]);
        tc_commit(&o_done[j & 1]);
      }
      if (!ok) fail();
      tc_commit(&drain);  // every MMA of this thread is done before tensor memory is freed
      if (!mbar_wait(&drain, 0)) fail();
    }
  } else if (works) {
    const uint32_t to = tl + kApTmO + half * 64;  // this thread's half of O
    const float c = a.scale_log2;
    float m_ref = -INFINITY, lsum = 0.f;
    bool ok = true;
    // exchange k of the pair: both halves have written xch[k & 1]
    auto pair_done = [&](int k) {
      tc_fence_before();
      mbar_arrive(&pair_bar[q]);
      const bool r = __all_sync(0xffffffffu, mbar_wait(&pair_bar[q], k & 1));
      tc_fence_after();
      return r;
    };
    for (int j = 0; j < T; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tb = tl + static_cast<uint32_t>((j & 1) * 128);
      uint32_t s0[32], s1[32];
      tc_ld32(s0, tb + half * 64);
      tc_ld32(s1, tb + half * 64 + 32);
      tc_wait_ld();
      float x[64];
#pragma unroll
      for (int k = 0; k < 64; ++k) x[k] = __uint_as_float(k < 32 ? s0[k] : s1[k - 32]);
      const int left = k1 - (k0 + j * kApKeys + half * 64);  // keys of this half inside the range
      if (left < 64) {
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (k >= left) x[k] = -INFINITY;
      }
      float mh[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) mh[k] = fmaxf(x[k], x[k + 32]);
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1)
#pragma unroll
        for (int k = 0; k < w; ++k) mh[k] = fmaxf(mh[k], mh[k + w]);
      xch[j & 1][half][v] = mh[0];
      if (!pair_done(j)) {
        ok = false;
        break;
      }
      const float mx = fmaxf(mh[0], xch[j & 1][half ^ 1][v]) * c;
      const bool move = mx > m_ref + kAmMargin;
      if (__any_sync(0xffffffffu, move)) {
        const float nref = move ? mx : m_ref;
        const float f = nref == m_ref ? 1.f : at_exp2(m_ref - nref);  // 0 on the first move
        lsum *= f;
        if (j > 0) {
          // O holds tiles 0 .. j - 1 once P_{j-1} V_{j-1} has completed
          if (!__all_sync(0xffffffffu, mbar_wait(&o_done[(j - 1) & 1], ((j - 1) >> 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += 32) {
            uint32_t o[32];
            tc_ld32(o, to + c0);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tc_st32(to + c0, o);
          }
        }
        m_ref = nref;
      }
      const float m = m_ref == -INFINITY ? 0.f : m_ref;  // no score seen yet: every term is 0
      // 32 at a time, over the scores that this warp has read
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t ph[16], pl[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float p0 = at_exp2(fmaf(x[32 * h + 2 * k], c, -m)), p1 = at_exp2(fmaf(x[32 * h + 2 * k + 1], c, -m));
          sum[k & 3] += p0 + p1;
          at_pack_split(p0, p1, &ph[k], &pl[k]);
        }
        tc_st16(tb + half * 32 + h * 16, ph);
        tc_st16(tb + 64 + half * 32 + h * 16, pl);
      }
      lsum += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[j & 1]);
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(&o_done[(T - 1) & 1], ((T - 1) >> 1) & 1))) ok = false;
    xch[T & 1][half][v] = lsum;
    if (!pair_done(T)) ok = false;  // (after a failure the pair may be out of step: bounded either way)
    float* so = reinterpret_cast<float*>(Ks);
    if (ok) {
      tc_fence_after();
      const long long at = static_cast<long long>(split) * a.batch * a.n_q + prow;
      if (have && half == 0) a.part_ml[at] = make_float2(m_ref, lsum + xch[T & 1][1][v]);
      // O through shared memory (the rings are done with), so that a warp writes
      // whole rows: 16-byte pieces a row apart from every lane kept the CTA 5 us
      // longer on its SM
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t o[32];
        tc_ld32(o, to + c0);
        tc_wait_ld();
        uint4* dst = reinterpret_cast<uint4*>(so + v * kApPitch + half * 64 + c0);
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    // The two warps of the lane quarter, each of which comes here whatever it gave up:
    // this barrier ends when their bounded waits have. (As a phase of pair_bar: 4 x 512
    // and 16 x 4096 take 0.2 us longer.)
    asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
    if (ok) {
#pragma unroll 4
      for (int r = q * 32 + half * 16; r < q * 32 + half * 16 + 16; ++r) {
        if (r >= nrows) break;
        const int row = row0 + r;
        const long long to_row = static_cast<long long>(split) * a.batch * a.n_q +
                                 static_cast<long long>(row / a.group) * a.n_q + g * a.group + row % a.group;
        *reinterpret_cast<float4*>(a.part_o + to_row * kApD + lane * 4) =
            *reinterpret_cast<const float4*>(so + r * kApPitch + lane * 4);
      }
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

}  // namespace wsg
