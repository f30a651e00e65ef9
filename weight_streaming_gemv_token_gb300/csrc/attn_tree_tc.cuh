// Attention of a step's rows on the 5th-generation tensor cores: bfloat16 queries and
// caches, head size 64 or 128, pages of 8 tokens and more. One CTA an SM, each an equal
// share of the line of key tiles (attn_tree_plan.h), row tiles of 128 rows.
//
// A row of the matrix products is a (token, query head) of the key/value head, one
// per tensor-memory lane. The CTA runs through its pieces one after the other, tiles
// of 128 keys in rings that do not stop between pieces:
//   warp 0      finds the CTA's share and cuts it into pieces, which it announces to
//               the others two or three tiles ahead; with warps 18 and 19 streams keys and
//               values, a box of 64 columns a page (128-byte swizzle), a lane a box, its table
//               entry read one tile ahead; each of the three arrives for every tile;
//   warp 1      one thread issues S_j = Q K_j^T one tile ahead, then O += P_j V_j with
//               P_j over the scores in tensor memory;
//   warps 2-17  four threads a row, 32 of the tile's keys each: masked, scaled scores,
//               reference maximum (moved only past a margin of 2^8, then O is rescaled in
//               place), probabilities as bfloat16 value + remainder, running sums. They
//               put the next piece's queries into tensor memory once the last scores of
//               a piece are read, so its first scores run while O is read. Every 16 tiles O
//               goes into a total (kTtSum). (Two threads a row: longer chains and twice the code to
//               fetch, 3,500 cycles a tile.)
// Tiles with drafted rows or the end of the keys: scores are masked row by row; value
// rows behind the end or of a page that is not there become 0 in shared memory, and so
// do values of drafted rows that are not finite, which are added afterwards to the rows
// that see them (0 times such a value would reach the others).
//
// Tensor memory (512 columns): scores / probabilities at 0 and 128, O at 256, Q at
// 384. The products of a tile of head size 128 take 24 x 64 cycles for any number of
// rows, its 64 KB at the SM's share of the measured bandwidth 2,700 at 1.85 GHz: bound
// by memory for up to 128 rows a head. Measured (16 query heads over 8, all requests as long as
// said): 32 x 64 rows x 16,384 tokens 373 us (5.8 TB/s), 48 single tokens x 7,000 219 (6.3 TB/s),
// 8 x 16 rows x 4,096 37.4.
//
// Every wait is bounded; on a timeout the CTA records ERR_TC_TIMEOUT, stops, waits
// for its issued MMAs and copies and frees its tensor memory.
#pragma once
#include "attn_tree.cuh"
#include "tc_attn_util.cuh"

namespace wsg {

constexpr int kTtSoft = 16;  // warps of the softmax
constexpr int kTtLoaders = 3;  // warps that issue copies: warp 0 and those behind the softmax's
constexpr int kTtThreads = 32 * (1 + kTtSoft + kTtLoaders), kTtRows = 128;
constexpr int kTtPieces = 8;  // pieces announced: the rings hold the tiles of fewer
constexpr uint32_t kTtTmO = 256, kTtTmQ = 384, kTtTmTotal = 448;
constexpr int kTtStage = 32 * 12;  // floats of a warp's way to memory: 32 rows of 32 bytes and 16 more
// Tiles whose products are summed in the matrix instructions. These cut sums off where an addition
// would round, always towards 0 (half a unit or less of 2^-23, 16 instructions a tile): over 16,384
// keys 5.7e-5 of a result, and results next to a border of bfloat16 rounded to its other side. 16
// tiles lose some 3.6e-6, less than probabilities in 16 bits do (4.4e-6); their sums are added up
// rounded, behind the last one's product (32 x 64 rows x 16,384 tokens 349 us without and 373 with
// it, 48 single tokens x 7,000 207 and 219; every 32 tiles 364 and 214, every 8 396 and 228).
constexpr int kTtSum = 16;

template <int D>
struct TtGeom {
  static constexpr int BOXES = D / 64;                // 64 columns each
  static constexpr uint32_t BOX = kAtKeys * 128;      // bytes of 128 keys' columns
  static constexpr uint32_t TILE = BOXES * BOX;
  static constexpr int STAGES = 3;                    // of keys, and of values
  static constexpr size_t SMEM = 2 * STAGES * TILE + kTtSoft * kTtStage * 4 + 1024;
};

// A tile's values in shared memory, a quarter of a row a thread (whole 128-byte lines, so
// the swizzle does not matter): rows behind k1 or of a missing page become 0, and so do
// values that are not finite of rows from n on; whether there were any. (Not inlined: its
// addresses would cost the main loop registers.)
template <int D>
__device__ __noinline__ bool tt_mend(unsigned char* tile, int tk, int n, int k1, uint32_t holes, int page_shift) {
  const int at = threadIdx.x - 64, row = at >> 2, key = tk + row;
  constexpr int N = D / 32;  // 16-byte pieces of a quarter
  unsigned char* line = tile + row * 128 + (D == 128 ? (at >> 1 & 1) * TtGeom<D>::BOX + (at & 1) * 64 : (at & 3) * 32);
  bool odd = false;
  if (key >= k1 || (holes >> (row >> page_shift) & 1u)) {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(line)[(i + row) & (N - 1)] = make_uint4(0, 0, 0, 0);
  } else if (key >= n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4* at16 = reinterpret_cast<uint4*>(line) + ((i + row) & (N - 1));
      const uint4 w = *at16;
      const uint4 z = make_uint4(at_finite2(w.x), at_finite2(w.y), at_finite2(w.z), at_finite2(w.w));
      if ((z.x ^ w.x) | (z.y ^ w.y) | (z.z ^ w.z) | (z.w ^ w.w)) *at16 = z, odd = true;
    }
  }
  return odd;
}

// Pairs of floats for the two-wide float32 instructions.
using TtPair = unsigned long long;
__device__ __forceinline__ TtPair tt_pair(float x, float y) {
  TtPair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ void tt_unpair(TtPair p, float* x, float* y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(p)); }
__device__ __forceinline__ TtPair tt_fma(TtPair a, TtPair b, TtPair c) {
  TtPair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ TtPair tt_add(TtPair a, TtPair b) {
  TtPair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ TtPair tt_sub(TtPair a, TtPair b) {
  TtPair d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// A pair as bfloat16 value and remainder pairs (at_pack_split).
__device__ __forceinline__ void tt_split(TtPair p, uint32_t* hi, uint32_t* lo) {
  float x, y;
  tt_unpair(p, &x, &y);
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  float rx, ry;
  tt_unpair(tt_sub(p, tt_pair(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u))), &rx, &ry);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(*lo) : "f"(ry), "f"(rx));
  *hi = h;
}
__device__ __forceinline__ float tt_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float tt_max3(uint32_t a, uint32_t b, uint32_t c) {
  return tt_max3(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c));
}

// N registers from or to this warp's lanes of tensor memory.
template <int N>
__device__ __forceinline__ void tt_ld(uint32_t (&v)[N], uint32_t at) {
  if constexpr (N == 32)
    tc_ld32(v, at);
  else
    tc_ld16(v, at);
}
template <int N>
__device__ __forceinline__ void tt_st(uint32_t at, const uint32_t (&v)[N]) {
  if constexpr (N == 32)
    tc_st32(at, v);
  else if constexpr (N == 16)
    tc_st16(at, v);
  else
    tc_st8(at, v);
}

// Adds to a thread's part of O, at `to` in tensor memory, the values of drafted rows that
// its row sees and that are not finite (which makes the sums not finite). One warp.
template <int D>
__device__ __noinline__ void tt_odd(const AtArgs& p, const AtPiece& x, uint32_t to, int sl, bool have, int token) {
  const AmArgs& a = p.a;
  const int32_t* trow = a.table + static_cast<long long>(x.s) * a.pool.width;
  for (int c0 = 0; c0 < D / 4; c0 += 16) {
    uint32_t o[16];
    tc_ld16(o, to + c0);
    tc_wait_ld();
    for (int key = max(x.k0, x.n); have && key < x.k1; ++key) {
      if (!(at_seen(p, x.begin, token, key - x.n) & 1u)) continue;
      const int page = page_of(a.pool, trow, key);
      if (page < 0) continue;
      const uint16_t* src = static_cast<const uint16_t*>(a.vp) + pool_row(a.pool, page, x.g, key) * D + sl * (D / 4) + c0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float y = bf16_to_f32(src[k]);
        if ((__float_as_uint(y) & 0x7F800000u) == 0x7F800000u) o[k] = __float_as_uint(__uint_as_float(o[k]) + y);
      }
    }
    __syncwarp();
    tc_st16(to + c0, o);
    tc_wait_st();
  }
}

// A thread's part of O over a piece's tiles but the last kTtSum or fewer: 16 columns in tensor
// memory at `at`, of D = 128 12 more in the warp's way to memory `so`; keep[0 .. 3]: the last 4, and
// keep[4] the total's reference. JOIN: O at `to`, whose reference is m, becomes the whole sum;
// otherwise the total takes O in (first: becomes it). One warp. (Not inlined, and not from within the
// loop over tiles: pieces that never come here would take 5 to 9% longer.)
template <int D, bool JOIN>
__device__ __noinline__ void tt_total(uint32_t to, uint32_t at, float* so, float* keep, float m, bool first) {
  const int lane = threadIdx.x & 31;
  const float ref = first ? m : keep[4], f = ref == m ? 1.f : at_exp2(ref - m);
#pragma unroll
  for (int c0 = 0; c0 < D / 4; c0 += 16) {
    uint32_t o[16], x[16];
    tc_ld16(o, to + c0);
    if (c0 == 0) {
      tc_ld16(x, at);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = first ? 0u : __float_as_uint(k < 12 ? so[k * 32 + lane] : keep[k - 12]);
    }
    tc_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = first ? o[k] : __float_as_uint(fmaf(__uint_as_float(x[k]), f, __uint_as_float(o[k])));
    if (JOIN) {
      tc_st16(to + c0, x);
    } else if (c0 == 0) {
      tc_st16(at, x);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k < 12)
          so[k * 32 + lane] = __uint_as_float(x[k]);
        else
          keep[k - 12] = __uint_as_float(x[k]);
      }
    }
  }
  tc_wait_st();
  keep[4] = m;
}

// The total takes O in once the product before, which `bar` tells, has completed. Whether it has.
template <int D>
__device__ __noinline__ bool tt_fold(uint64_t* bar, uint32_t phase, uint32_t to, uint32_t at, float* so, float* keep, float m, bool first) {
  if (!__all_sync(0xffffffffu, mbar_wait(bar, phase))) return false;
  tc_fence_after();
  tt_total<D, false>(to, at, so, keep, m, first);
  return true;
}

// pk, pv: the prefix as [n_kv][plen][D] in boxes of 128 x 64; kp, vp: the pools as
// [pages * n_kv][page][D] in boxes of min(page, 128) x 64.
template <int D>
__global__ void __launch_bounds__(kTtThreads, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap pk, const __grid_constant__ CUtensorMap pv,
                        const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp,
                        const __grid_constant__ AtArgs p) {
  using G = TtGeom<D>;
  constexpr int PART = D / 4, STAGES = G::STAGES;  // columns of O a thread holds
  extern __shared__ __align__(1024) unsigned char tt_raw[];
  unsigned char* Ks = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tt_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* Vs = Ks + STAGES * G::TILE;
  float* So = reinterpret_cast<float*>(Vs + STAGES * G::TILE);
  __shared__ AtPiece s_piece[kTtPieces], s_dry;
  __shared__ uint32_t s_holes[kTtPieces];  // by tile: pages that are missing
  __shared__ __align__(8) uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_done[2], q_full, o_free, drain, row_bar[4], told[kTtPieces];
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail, s_put[kTtLoaders][2];
  // whether a piece had drafted values that are not finite, by its parity: a warp may be at the piece behind while another
  // has yet to read what this one had (not two behind: every warp puts each piece's queries)
  __shared__ int s_odd[2];
  __shared__ float xch[2][4][kTtRows];
  const AmArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* vfail = &s_fail;
  volatile int* vodd = s_odd;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&k_full[s], kTtLoaders), mbar_init(&k_empty[s], 1), mbar_init(&v_full[s], kTtLoaders), mbar_init(&v_empty[s], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&s_full[b], 1), mbar_init(&p_full[b], kTtSoft), mbar_init(&o_done[b], 1);
    mbar_init(&q_full, kTtSoft);
    mbar_init(&o_free, kTtSoft);
    mbar_init(&drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&row_bar[i], 4);
    for (int i = 0; i < kTtPieces; ++i) mbar_init(&told[i], 1);
    s_fail = 0;
    s_odd[0] = s_odd[1] = -1;
    s_dry = AtPiece{};
    s_dry.prefix = true;
    s_dry.nrows = kTtRows;
    s_dry.k1 = kAtKeys;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  auto fail = [&]() {
    *vfail = 1;
    atomicOr(a.err, ERR_TC_TIMEOUT);
  };
  const int shift = a.pool.shift, page_shift_ = min(shift, kAtKeyShift), tile_pages = kAtKeys >> page_shift_;

  if (warp == 0 || warp > 1 + kTtSoft) {
    // ---- the share, keys and values ----
    const int who = warp == 0 ? 0 : warp - 1 - kTtSoft;  // which of the loaders
    pdl_wait();
    pdl_trigger();
    AtWalk walk;
    if (who == 0) walk = at_start(p);
    int j = 0, keys = 0, values = 0;  // tiles so far; those whose keys, values this loader has asked for
    bool ok = true;
    AtPiece pc{};
    // this loader's boxes are numbers who, who + loaders, .. of (page, 64 columns); this lane's one
    const int unit = lane * kTtLoaders + who, unit_page = unit / G::BOXES, unit_box = unit % G::BOXES;
    // the table's entry for a page of the tile at key tk, -1 where there is none to read
    auto entry = [&](int tk, int page) -> int32_t {
      const int at = tk + (page << page_shift_);
      return pc.prefix || page >= tile_pages || at >= pc.k1
                 ? -1
                 : a.table[static_cast<long long>(pc.s) * a.pool.width + (at >> shift)];
    };
    for (int piece = 0; ok; ++piece) {
      if (who == 0) {
        pc = walk.next(p);
        if (lane == 0) {
          s_piece[piece % kTtPieces] = pc;
          mbar_arrive(&told[piece % kTtPieces]);
        }
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&told[piece % kTtPieces], (piece / kTtPieces) & 1))) {
          ok = false;
          break;
        }
        pc = s_piece[piece % kTtPieces];
      }
      if (pc.tiles == 0) break;
      if (who == 1) {
        // the queries on their way, ahead of the keys that fill the memory's queues
        const int per = p.cut.group * D * 2, t0 = pc.m0 / a.group, t1 = (pc.m0 + pc.nrows - 1) / a.group;
        const char* q0 = static_cast<const char*>(a.q) + (a.q_stride * pc.begin + static_cast<long long>(pc.g) * a.group * D) * 2;
        const int lines = (per + 127) / 128;
        for (int i = lane; i < (t1 - t0 + 1) * lines; i += 32) {
          const int t = i / lines;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q0 + a.q_stride * 2 * (t0 + t) + (i - t * lines) * 128));
        }
      }
      int32_t e = entry(pc.k0, unit_page), all = who == 0 ? entry(pc.k0, lane) : -1;
      for (int i = 0; i < pc.tiles; ++i, ++j) {
        const int tk = pc.k0 + i * kAtKeys, st = j % STAGES;
        const bool there = e >= 0 && e < a.pool.num_pages;
        const int plane = e * a.n_kv + pc.g, y = shift > kAtKeyShift ? tk & ((1 << shift) - 1) : 0;
        const uint32_t part = 128u << page_shift_;  // bytes of a page's columns
        const bool mine = pc.prefix ? unit < G::BOXES : there;  // this lane copies a box
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * (pc.prefix ? G::BOX : part);
        uint32_t holes = 0;
        if (who == 0) {
          const bool wanted = !pc.prefix && lane < tile_pages && tk + (lane << page_shift_) < pc.k1;
          holes = __ballot_sync(0xffffffffu, wanted && !(all >= 0 && all < a.pool.num_pages));
        }
        if (i + 1 < pc.tiles) {
          e = entry(tk + kAtKeys, unit_page);
          if (who == 0) all = entry(tk + kAtKeys, lane);
        }
        // (every loader arrives for every tile: none falls so far behind that it mistakes a barrier's phase)
        auto load = [&](unsigned char* dst, const CUtensorMap* pre, const CUtensorMap* pages, uint64_t* bar) {
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (!mine) return;
          if (pc.prefix)
            tma_load_3d_map(dst + unit * G::BOX, pre, unit * 64, tk, pc.g, bar);
          else
            tma_load_3d_map(dst + unit_box * G::BOX + unit_page * part, pages, unit_box * 64, y, plane, bar);
        };
        if (j >= STAGES && !__all_sync(0xffffffffu, mbar_wait(&k_empty[st], ((j / STAGES) - 1) & 1))) {
          ok = false;
          break;
        }
        if (who == 0 && lane == 0) {
          s_holes[j % kTtPieces] = holes;
          if (holes) atomicOr(a.err, ERR_BAD_PAGE);
        }
        load(Ks + st * G::TILE, &pk, &kp, &k_full[st]);
        keys = j + 1;
        if (j >= STAGES && !__all_sync(0xffffffffu, mbar_wait(&v_empty[st], ((j / STAGES) - 1) & 1))) {
          ok = false;
          break;
        }
        load(Vs + st * G::TILE, &pv, &vp, &v_full[st]);
        values = j + 1;
        if (__any_sync(0xffffffffu, *vfail)) {
          ok = false;
          break;
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (who == 0 && p.prefix_tiles == 0) {
      if (!ok) {  // the share's records all the same, for the join: nothing of its cut segment
        while (walk.next(p).tiles > 0) {
        }
        walk.seam_seg = -1;
        walk.seam = AtSeam{};
      }
      at_seams(p, walk);
    }
    // the last copies into each stage have landed before the CTA may end; after a failure a loader first
    // arrives for the tiles (STAGES at most) that it did not come to and another did
    if (lane == 0) s_put[who][0] = keys, s_put[who][1] = values;
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kTtLoaders) : "memory");
    if (lane == 0) {
      for (int w = 0; w < 2; ++w) {
        int top = 0;
        for (int i = 0; i < kTtLoaders; ++i) top = max(top, s_put[i][w]);
        uint64_t* full = w ? v_full : k_full;
        for (int i = s_put[who][w]; i < top; ++i) mbar_arrive(&full[i % STAGES]);
        for (int s = 0; s < STAGES; ++s)
          if (who == 0 && s < top && !mbar_wait(&full[s], ((top - 1 - s) / STAGES) & 1, kLandLimitNs)) fail();
      }
    }
  } else if (warp == 1) {
    pdl_wait();  // (the limits of its waits do not count the time of the stream's previous kernel)
    if (lane == 0) {
      constexpr uint32_t idS = tc_idesc(kTtRows, kAtKeys);
      constexpr uint32_t idO = tc_idesc(kTtRows, D) | (1u << 16);  // B (values) MN-major
      int j = 0, piece = 0;
      bool ok = true, issued = false;
      auto issue_s = [&](int i) -> bool {
        const int s = i % STAGES;
        if (!mbar_wait(&k_full[s], (i / STAGES) & 1)) return false;
        tc_fence_after();
        issued = true;
        const uint32_t kb = smem_u32(Ks + s * G::TILE), d = tmem + static_cast<uint32_t>((i & 1) * 128);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_f16_ts(d, tmem + kTtTmQ + kk * 8, tc_desc_sw128(kb + (kk >> 2) * G::BOX + (kk & 3) * 32), idS, kk != 0);
        tc_commit(&k_empty[s]);
        tc_commit(&s_full[i & 1]);
        return true;
      };
      for (; ok; ++piece) {
        if (!mbar_wait(&told[piece % kTtPieces], (piece / kTtPieces) & 1)) {
          ok = false;
          break;
        }
        const int T = s_piece[piece % kTtPieces].tiles;
        if (T == 0) break;
        if (!mbar_wait(&q_full, piece & 1) || !issue_s(j)) {
          ok = false;
          break;
        }
        for (int t = 0; t < T; ++t, ++j) {
          // S_{j+1} replaces P_{j-1}: it is issued after P_{j-1} V_{j-1} and runs after it
          if (t + 1 < T && !issue_s(j + 1)) {
            ok = false;
            break;
          }
          const int s = j % STAGES;
          if (!mbar_wait(&p_full[j & 1], (j >> 1) & 1) || !mbar_wait(&v_full[s], (j / STAGES) & 1) ||
              (t == 0 && piece > 0 && !mbar_wait(&o_free, (piece - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t vb = smem_u32(Vs + s * G::TILE), pb = tmem + static_cast<uint32_t>((j & 1) * 128);
#pragma unroll
          for (int kk = 0; kk < kAtKeys / 16; ++kk) {
            const uint64_t db = tc_desc_sw128_mn(vb + kk * 2048, G::BOX, 1024);
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc_mma_f16_ts(tmem + kTtTmO, pb + part * 64 + kk * 8, db, idO, (t % kTtSum | kk | part) != 0);
          }
          tc_commit(&v_empty[s]);
          tc_commit(&o_done[j & 1]);
        }
        if (*vfail) ok = false;
      }
      if (!ok) fail();
      if (issued) {  // every MMA of this thread is done before tensor memory is freed
        tc_commit(&drain);
        if (!mbar_wait(&drain, 0, kLandLimitNs)) fail();
      }
    }
  } else {
    const int q = warp & 3, sl = (warp - 2) >> 2;  // lane quarter; which of the row's four threads
    const int v = q * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);  // this warp's lanes
    const uint32_t to = tl + kTtTmO + sl * PART;                       // this thread's part of O
    const float c = a.scale_log2;
    float* so = So + (warp - 2) * kTtStage;
    int j = 0, ex = 0;  // tiles, exchanges among a row's threads so far
    bool ok = true;
    // Piece -1 is made up: a tile of whatever tensor memory holds, whose result goes
    // nowhere. It has the code of tiles and results fetched while the stream's previous kernel ends
    // (behind the first keys' copies, which fill the memory's queues, that takes 5 us).
    bool dry = true;
    float keep[5];  // of the total over earlier tiles
    const uint32_t tt = tl + kTtTmTotal + sl * 16;
    auto row_done = [&]() {
      tc_fence_before();
      __syncwarp();
      if (dry) return true;
      if (lane == 0) mbar_arrive(&row_bar[q]);
      const bool r = __all_sync(0xffffffffu, mbar_wait(&row_bar[q], ex & 1));
      tc_fence_after();
      ++ex;
      return r;
    };
    // Waits for piece number i; its tiles.
    auto piece_at = [&](int i) -> int {
      if (!__all_sync(0xffffffffu, mbar_wait(&told[i % kTtPieces], (i / kTtPieces) & 1))) {
        ok = false;
        return 0;
      }
      return s_piece[i % kTtPieces].tiles;
    };
    // this thread's part of its row of the piece's queries into tensor memory
    auto queries = [&](const AtPiece& x) {
      const int nrows = x.nrows;
      if (q * 32 < nrows) {
        uint32_t qr[PART / 2];
#pragma unroll
        for (int i = 0; i < PART / 2; ++i) qr[i] = 0;
        if (v < nrows) {
          const int m = x.m0 + v, token = m / a.group;
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + a.q_stride * (x.begin + token) +
                                (x.g * a.group + m - token * a.group) * D + sl * PART;
          if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
            for (int i = 0; i < PART / 8; ++i) {
              const uint4 w = reinterpret_cast<const uint4*>(src)[i];
              qr[4 * i] = w.x, qr[4 * i + 1] = w.y, qr[4 * i + 2] = w.z, qr[4 * i + 3] = w.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < PART / 2; ++i) qr[i] = src[2 * i] | (static_cast<uint32_t>(src[2 * i + 1]) << 16);
          }
        }
        if (a.q_sign != 1) {
#pragma unroll
          for (int i = 0; i < PART / 2; ++i) qr[i] = a.q_sign == 0 ? 0u : qr[i] ^ 0x80008000u;
        }
        tt_st(tl + kTtTmQ + sl * (PART / 2), qr);
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
    };
    if (warp == 1 + kTtSoft && p.prefix_tiles > 0) {
      pdl_wait();
      at_records(p);  // (while the first keys are on their way)
    }
    int T = 1;
#pragma unroll 1
    for (int piece = -1; T > 0; ++piece) {
      const AtPiece& cur = dry ? s_dry : s_piece[piece % kTtPieces];
      const bool works = q * 32 < cur.nrows, have = v < cur.nrows && !dry;
      const int m_row = cur.m0 + min(v, cur.nrows - 1), token = m_row / a.group;
      const int k0 = cur.k0, k1 = cur.k1;
      const int plain = cur.prefix ? k1 : min(cur.n, k1);  // keys before this one are seen by every row
      float m_ref = -INFINITY, lsum = 0.f;
      int t = 0;
      auto tile = [&]() -> bool {
        const int tk = k0 + t * kAtKeys;
        if (!dry && !__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j >> 1) & 1))) {
          return false;
        }
        tc_fence_after();
        const uint32_t holes = dry ? 0u : s_holes[j % kTtPieces];
        const bool special = holes || (tk + kAtKeys > plain && !cur.prefix);
        if (works) {
          const uint32_t tb = tl + static_cast<uint32_t>((j & 1) * 128);
          uint32_t s[32];
          tc_ld32(s, tb + sl * 32);
          tc_wait_ld();
          const int first = tk + sl * 32;
          if (holes || first + 32 > plain) {
            uint32_t see = cur.prefix ? 0xffffffffu : at_seen(p, cur.begin, token, first - cur.n);
            if (k1 - first < 32) see &= k1 > first ? (1u << (k1 - first)) - 1u : 0u;
            if (holes)
              for (int i = 0; i < 4; ++i)
                if (holes >> ((sl * 32 + 8 * i) >> page_shift_) & 1u) see &= ~(0xffu << (8 * i));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(see >> k & 1u)) s[k] = 0xff800000u;  // -inf
          }
          float mh[11];  // three at a time: 32 -> 11 -> 4 -> 2 -> 1
#pragma unroll
          for (int k = 0; k < 10; ++k) mh[k] = tt_max3(s[3 * k], s[3 * k + 1], s[3 * k + 2]);
          mh[10] = fmaxf(__uint_as_float(s[30]), __uint_as_float(s[31]));
#pragma unroll
          for (int k = 0; k < 3; ++k) mh[k] = tt_max3(mh[3 * k], mh[3 * k + 1], mh[3 * k + 2]);
          mh[0] = fmaxf(tt_max3(mh[0], mh[1], mh[2]), fmaxf(mh[9], mh[10]));
          float(&x)[4][kTtRows] = xch[ex & 1];
          x[sl][v] = mh[0];
          if (!row_done()) {
            return false;
          }
          const float mx = fmaxf(fmaxf(x[0][v], x[1][v]), fmaxf(x[2][v], x[3][v])) * c;
          const bool move = mx > m_ref + kAmMargin;
          if (__any_sync(0xffffffffu, move)) {
            const float nref = move ? mx : m_ref;
            const float f = nref == m_ref ? 1.f : at_exp2(m_ref - nref);  // 0 on the first move
            lsum *= f;
            if (t > 0) {
              // O holds the piece's tiles before this one once P_{j-1} V_{j-1} has completed
              if (!__all_sync(0xffffffffu, mbar_wait(&o_done[(j - 1) & 1], ((j - 1) >> 1) & 1))) {
                return false;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < PART; c0 += 16) {  // (32 at a time would spill the scores)
                uint32_t o[16];
                tc_ld16(o, to + c0);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc_st16(to + c0, o);
              }
            }
            m_ref = nref;
          }
          const float m = m_ref == -INFINITY ? 0.f : m_ref;  // no score seen yet: every term is 0
          const TtPair c2 = tt_pair(c, c), m2 = tt_pair(-m, -m);
          TtPair sum = tt_pair(0.f, 0.f);
          // over the scores, which all four threads of the row have read
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t ph[8], pl[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float x0, x1;
              tt_unpair(tt_fma(tt_pair(__uint_as_float(s[16 * h + 2 * k]), __uint_as_float(s[16 * h + 2 * k + 1])), c2, m2), &x0, &x1);
              const TtPair e = tt_pair(at_exp2(x0), at_exp2(x1));
              sum = tt_add(sum, e);
              tt_split(e, &ph[k], &pl[k]);
            }
            tc_st8(tb + sl * 16 + 8 * h, ph);
            tc_st8(tb + 64 + sl * 16 + 8 * h, pl);
          }
          float s0, s1;
          tt_unpair(sum, &s0, &s1);
          lsum += s0 + s1;
          tc_wait_st();
        }
        if (special) {
          const int st = j % STAGES;
          if (!__all_sync(0xffffffffu, mbar_wait(&v_full[st], (j / STAGES) & 1))) {
            return false;
          }
          if (tt_mend<D>(Vs + st * G::TILE, tk, cur.n, k1, holes, page_shift_)) vodd[piece & 1] = piece + 1;
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !dry) mbar_arrive(&p_full[j & 1]);
        return true;
      };
      while (true) {
        for (const int end = min(T, t + kTtSum); ok && t < end; ++t, ++j) ok = tile();
        if (!ok || t >= T) break;
        // O into the total once the last product has completed; the next one starts it anew
        if (works) {
          if (!(ok = tt_fold<D>(&o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, to, tt, so, keep, m_ref, t == kTtSum))) break;
        }
      }
      if (!ok) break;
      if (dry) {
        pdl_wait();
        pdl_trigger();
        j = 0;
      }
      T = piece_at(piece + 1);
      if (T > 0) queries(s_piece[(piece + 1) % kTtPieces]);
      // ---- the piece's result ----
      if (!dry && !__all_sync(0xffffffffu, mbar_wait(&o_done[(j - 1) & 1], ((j - 1) >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (works) {
        float(&x)[4][kTtRows] = xch[ex & 1];
        x[sl][v] = lsum;
        if (!row_done()) {
          ok = false;
          break;
        }
        lsum = (x[0][v] + x[1][v]) + (x[2][v] + x[3][v]);
        if (t > kTtSum) tt_total<D, true>(to, tt, so, keep, m_ref, false);
        if (vodd[piece & 1] == piece + 1) tt_odd<D>(p, cur, to, sl, have, token);
        const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;  // a NaN sum stays one
        if (sl == 0 && have) {
          if (!cur.whole)
            a.part_ml[cur.id * kTtRows + v] = make_float2(m_ref, lsum);
          else if (p.lse)
            p.lse[static_cast<long long>(cur.begin + token) * a.n_q + cur.g * a.group + m_row - token * a.group] =
                lsum == 0.f ? -INFINITY : (m_ref + log2f(lsum)) * 0.69314718f;
        }
        // 32 bytes of every row at a time through shared memory, so that whole sectors leave: two lanes a row
        auto leave = [&](const uint32_t(&w)[8], auto put) {
          __syncwarp();  // the part before this one has left
          uint4* dst = reinterpret_cast<uint4*>(so + lane * 12);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = h * 16 + (lane >> 1);
            if (q * 32 + r < cur.nrows && !dry) put(q * 32 + r, *reinterpret_cast<const uint4*>(so + r * 12 + (lane & 1) * 4));
          }
        };
#pragma unroll 1
        for (int c0 = 0; c0 < PART; c0 += 16) {
          uint32_t o[16];
          tc_ld16(o, to + c0);
          tc_wait_ld();
          if (c0 + 16 >= PART) {  // O is read: the next piece may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && !dry) mbar_arrive(&o_free);
          }
          if (cur.whole) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(w[k])
                  : "f"(__uint_as_float(o[2 * k + 1]) * inv), "f"(__uint_as_float(o[2 * k]) * inv));
            leave(w, [&](int row, uint4 x) {
              const int m = cur.m0 + row, tok = m / a.group;
              uint16_t* dst = static_cast<uint16_t*>(p.out) + p.out_stride * (cur.begin + tok) +
                              static_cast<long long>(cur.g * a.group + m - tok * a.group) * D + sl * PART + c0 + (lane & 1) * 8;
              if (p.out16) {
                *reinterpret_cast<uint4*>(dst) = x;
              } else {
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = static_cast<uint16_t>(y[k >> 1] >> (16 * (k & 1)));
              }
            });
          } else {
            float* part = a.part_o + cur.id * kTtRows * D + sl * PART + c0 + (lane & 1) * 4;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t w[8] = {o[8 * b], o[8 * b + 1], o[8 * b + 2], o[8 * b + 3], o[8 * b + 4], o[8 * b + 5], o[8 * b + 6], o[8 * b + 7]};
              leave(w, [&](int row, uint4 x) { *reinterpret_cast<uint4*>(part + row * D + 8 * b) = x; });
            }
          }
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free);
      }
      if (__any_sync(0xffffffffu, *vfail)) ok = false;
      if (!ok) break;
      dry = false;
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

}  // namespace wsg
