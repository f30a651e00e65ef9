// The second kernel of attn_shared_prefix where attn_prefix_tc_kernel takes the
// prefix and the branches' own keys are few: a CTA per (branch, key/value head)
// attends to the branch's own pages (attn_rows.cuh: ArCore, ArCopy) while the
// prefix kernel runs on the same SM, then waits for that kernel, joins its own
// result with the prefix's partial results of the same rows and writes the output.
// So no third launch waits for the second (16 x 4096 + 256 keys: 16.4 us with a
// join kernel, 11.7 like this).
#pragma once
#include "attn_rows.cuh"

namespace wsg {

struct AoArgs {
  int prefix_slots;
  void* out;
  long long out_stride;
  float* lse;
};

// Grid: batch * n_kv CTAs of four warps; warp w takes blocks w, w + 4, ... NB: rows
// of a branch (8, or 16 for groups over 8).
template <int NB>
__global__ void __maxnreg__(152) attn_own_kernel(const AmArgs a, const AoArgs j) {
  constexpr int DP = 128, WARPS = 4;
  using G = ArGeom<DP, NB, WARPS>;
  extern __shared__ __align__(128) unsigned char am_raw[];
  __shared__ float s_m[WARPS][NB], s_l[WARPS][NB];
  __shared__ float4 s_x[WARPS][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.n_kv, g = blockIdx.x % a.n_kv;
  if (a.first) pdl_wait();  // no prefix: nothing has waited for the stream's previous kernel
  pdl_trigger();
  const int n = a.len[b];
  if (n < 0) {
    pdl_wait();
    return;
  }
  int held = n;
  if (held > page_capacity(a.pool)) {
    held = static_cast<int>(page_capacity(a.pool));
    if (g == 0 && tid == 0) atomicOr(a.err, ERR_BAD_PAGE);
  }
  unsigned char* mine = am_raw + warp * G::PER_WARP;
  const uint32_t ring = smem_u32(mine);
  const ArCopy<DP> copy(a.d, mine);
  const int32_t* trow = a.table + static_cast<long long>(b) * a.pool.width;
  const int nblk = (held + 15) / 16;
  // the table's entry of a block's page, read one block before its keys are requested
  auto entry = [&](int blk) { return blk < nblk && a.pool.shift >= 4 ? trow[blk * 16 >> a.pool.shift] : 0; };
  auto request = [&](int stage, int blk, int32_t e) { return copy.pages(a, stage, trow, e, g, blk * 16, min(16, held - blk * 16)); };
  int32_t e0 = entry(warp), e1 = entry(warp + WARPS);
  uint32_t ok = 0;
  if (warp < nblk) ok = request(0, warp, e0);
  am_commit();
  ArCore<uint16_t, DP, 1, NB> core;
  const long long q0 = a.q_stride * b + static_cast<long long>(g) * a.group * a.d;
  core.load(a, a.group, [&](int r) { return q0 + static_cast<long long>(r) * a.d; });
  int stage = 0;
  for (int blk = warp; blk < nblk; blk += WARPS, stage ^= 1) {
    __syncwarp();  // every lane is done with the block before this one
    const uint32_t next = blk + WARPS < nblk ? request(stage ^ 1, blk + WARPS, e1) : 0;
    am_commit();
    e1 = entry(blk + 2 * WARPS);
    am_wait<1>();
    __syncwarp();  // this block has landed for every lane
    core.consume(ring + stage * 2 * G::TILE, ok, a.scale_log2);
    ok = next;
  }
  am_wait<0>();
  core.finish();
  __syncwarp();
  // this warp's result in the place of its ring
  float* o = reinterpret_cast<float*>(mine);
#pragma unroll
  for (int t = 0; t < NB / 8; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = t * 8 + 2 * (lane & 3) + i;
      if (r >= a.group) continue;
      if (lane < 4) s_m[warp][r] = core.m[t][i], s_l[warp][r] = core.l[t][i];
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        o[r * DP + k * 16 + (lane >> 2)] = core.o[k][t][i];
        o[r * DP + k * 16 + 8 + (lane >> 2)] = core.o[k][t][2 + i];
      }
    }
  __syncthreads();
  pdl_wait();  // the prefix's partial results

  // join: `per` warps a row, which take its parts in turn (the four own ones, then
  // the prefix's slots), eight at a time; lane i holds elements 4 i .. 4 i + 3
  const int per = a.group >= 4 ? 1 : a.group >= 2 ? 2 : 4, parts = WARPS + j.prefix_slots;
  const long long total = static_cast<long long>(a.batch) * a.n_q;
  for (int r0 = 0; r0 < a.group; r0 += WARPS / per) {
    const int r = r0 + warp / per;
    const long long row = static_cast<long long>(b) * a.n_q + g * a.group + r;
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = warp % per; s0 < parts && r < a.group; s0 += 8 * per) {
      float2 p[8];
      float4 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int s = s0 + i * per;
        if (s < WARPS) {
          p[i] = make_float2(s_m[s][r], s_l[s][r]);
          y[i] = *reinterpret_cast<const float4*>(am_raw + s * G::PER_WARP + (r * DP + lane * 4) * 4);
        } else if (s < parts) {
          const long long at = (s - WARPS) * total + row;
          p[i] = a.part_ml[at];
          y[i] = *reinterpret_cast<const float4*>(a.part_o + at * DP + lane * 4);
        } else {
          p[i] = make_float2(-INFINITY, 0.f);
          y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      ar_merge8(p, y, &m, &l, &x);
    }
    if (per > 1) {  // the row's other warps
      __syncthreads();
      if (lane == 0) s_m[warp][NB - 1] = m, s_l[warp][NB - 1] = l;  // (groups under 4 leave row NB - 1 free)
      s_x[warp][lane] = x;
      __syncthreads();
      if (warp % per == 0) {
        float2 p[8];
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = make_float2(-INFINITY, 0.f);
          y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i > 0 && i < per) p[i] = make_float2(s_m[warp + i][NB - 1], s_l[warp + i][NB - 1]), y[i] = s_x[warp + i][lane];
        }
        ar_merge8(p, y, &m, &l, &x);
      }
    }
    if (r >= a.group || warp % per) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // a NaN sum stays one
    uint16_t* dst = static_cast<uint16_t*>(j.out) + j.out_stride * b + static_cast<long long>(g * a.group + r) * DP + lane * 4;
    uint32_t h[2];
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(x.y * inv), "f"(x.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(x.w * inv), "f"(x.z * inv));
    if ((reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
    }
    if (j.lse && lane == 0) j.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
  }
}

}  // namespace wsg
