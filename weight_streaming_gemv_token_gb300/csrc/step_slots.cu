// step_slots: block tables, slots, positions and ancestor masks of a step from the
// requests' lengths.
//
// Mathematics: with need_s = max(0, ceil((held_s + fresh_s) / page) - owned_s) and
// the inclusive sum C_s of the needs before and at s, request s is served iff
// need_s = 0 or C_s <= free, and its j-th new page is entry first + C_s - need_s + j
// of the ring. C never falls, so all that ask and come after one that is not served
// are not served either, and C_s - need_s is what the served ones before s took.
// Row i of a request: its ancestors by walking the parents up, at most 255 rows
// before it, which a block of 256 rows keeps in shared memory with the 256 before.
//
// Every CTA sums the lengths of all requests for itself (a block scan of 4096 at
// most), so one launch does without a wait between CTAs; then the CTAs share out
// the rows (one thread each) and the table's rows. Bound by latency: the lengths'
// loads, three scans, a lookup, the page's load. Measured: 5.1 us for one request of 8
// rows, 7.6 for 256 of 32 whose tables of 514 entries are copied.
#include "common.h"
#include "paging.h"
#include "ptx.cuh"
#include "spans.h"

namespace wsg {
namespace {

constexpr int kSlThreads = 256, kSlRequests = 4096, kSlTree = 256;

struct SlArgs {
  int requests, rows, num_pages, shift, width, base_pos, words;
  int tree_max;  // rows that a request may bring
  const int32_t *held, *fresh, *owned, *parents, *table;
  int32_t* ring;
  const int32_t* state;
  int32_t *new_table, *new_owned, *new_state, *row_start, *ctx_len, *seq, *pos;
  int64_t* slots;
  uint32_t* mask;
  int in_place;
  uint32_t* err;
};

// Exclusive sums over the block of one value a thread; *total: the sum of all.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSlThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kSlThreads) step_slots_kernel(const SlArgs a) {
  // of request s: its first row, and where its pages start among those given out (bit 31:
  // not served or ended) or, for an ended one, among those that come back
  extern __shared__ int32_t s_mem[];
  int32_t* s_row = s_mem;                      // [requests + 1]
  uint32_t* s_at = reinterpret_cast<uint32_t*>(s_mem + a.requests + 1);  // [requests]
  __shared__ long long s_warp[kSlThreads / 32];
  __shared__ int32_t s_parent[2 * kSlTree];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  uint32_t bad = 0;
  int first = a.state[0], count = a.state[1];
  if (first < 0 || count < 0 || count > a.num_pages || (first >= a.num_pages && (first > 0 || count > 0))) {
    bad |= ERR_BAD_PAGE;
    first = count = 0;
  }
  // ---- the requests' rows and pages ----
  const int per = (a.requests + kSlThreads - 1) / kSlThreads;
  const int lo = min(a.requests, tid * per), hi = min(a.requests, lo + per);
  auto rows_of = [&](int s) { return a.held[s] >= 0 ? max(0, a.fresh[s]) : 0; };
  auto owned_of = [&](int s) { return min(max(0, a.owned[s]), a.width); };
  long long mine = 0, total;
  for (int s = lo; s < hi; ++s) mine += rows_of(s);
  long long at = block_scan(mine, s_warp, &total);
  // pages that request s, whose rows start at `row`, asks for; -1: it cannot be served
  auto need_of = [&](int s, long long row) -> long long {
    const int held = a.held[s];
    if (held < 0) return 0;
    const int n = max(0, a.fresh[s]);
    const long long pages = (static_cast<long long>(held) + n + (1 << a.shift) - 1) >> a.shift;
    if (a.owned[s] < 0 || a.owned[s] > a.width || pages > a.width || row + n > a.rows) {
      bad |= ERR_BAD_PAGE;
      if (pages > a.width || row + n > a.rows) return -1;
    }
    if (n > a.tree_max) {
      bad |= ERR_BAD_TREE;
      return -1;
    }
    return max(0ll, pages - owned_of(s));
  };
  long long row = at, asks = 0, back = 0;
  for (int s = lo; s < hi; ++s) {
    asks += max(0ll, need_of(s, row));
    if (a.held[s] < 0) back += owned_of(s);
    row += rows_of(s);
  }
  long long asked, backs;
  long long ask_at = block_scan(asks, s_warp, &asked), back_at = block_scan(back, s_warp, &backs);
  row = at;
  long long given = 0;  // pages that this thread's requests take
  for (int s = lo; s < hi; ++s) {
    const long long need = need_of(s, row);
    s_row[s] = static_cast<int32_t>(min(row, static_cast<long long>(a.rows)));
    if (a.held[s] < 0) {
      s_at[s] = 0x80000000u | static_cast<uint32_t>(min(back_at, 0x7fffffffll));
      back_at += owned_of(s);
    } else {
      const bool served = need >= 0 && (need == 0 || ask_at + need <= count);
      s_at[s] = served ? static_cast<uint32_t>(need == 0 ? 0 : ask_at) : 0x80000000u;
      if (served) given += need;
      ask_at += max(0ll, need);
    }
    row += rows_of(s);
  }
  if (tid == 0) s_row[a.requests] = static_cast<int32_t>(min(total, static_cast<long long>(a.rows)));
  long long all_given;
  block_scan(given, s_warp, &all_given);  // (its barriers also show s_row and s_at to all)
  const long long room = static_cast<long long>(a.num_pages) - count;
  if (backs > room) bad |= ERR_BAD_PAGE;
  const int returned = static_cast<int>(min(backs, room));
  auto ring_at = [&](long long i) { return static_cast<int>((first + i) % a.num_pages); };

  // ---- tables, lengths, the ring ----
  if (blockIdx.x == 0) {
    for (int s = tid; s <= a.requests; s += kSlThreads) a.row_start[s] = s_row[s];
    if (tid == 0) {
      a.new_state[0] = a.num_pages ? ring_at(all_given) : 0;
      a.new_state[1] = static_cast<int32_t>(count - all_given + returned);
    }
  }
  for (int s = blockIdx.x; s < a.requests; s += gridDim.x) {
    const int held = a.held[s], owned = owned_of(s);
    const bool served = !(s_at[s] >> 31);
    const long long pages = (static_cast<long long>(max(0, held)) + max(0, a.fresh[s]) + (1 << a.shift) - 1) >> a.shift;
    const int got = served ? static_cast<int>(max(0ll, pages - owned)) : 0;
    const uint32_t from = s_at[s] & 0x7fffffffu;
    const int32_t* old = a.table + static_cast<long long>(s) * a.width;
    int32_t* to = a.new_table + static_cast<long long>(s) * a.width;
    if (tid == 0) {
      a.ctx_len[s] = served ? held : -1;
      a.new_owned[s] = held < 0 ? 0 : owned + got;
    }
    if (held < 0)
      for (int j = tid; j < owned; j += kSlThreads)
        if (from + static_cast<long long>(j) < returned) a.ring[ring_at(count + from + static_cast<long long>(j))] = old[j];
    const int begin = a.in_place ? owned : 0, end = a.in_place ? owned + got : a.width;
    for (int j = begin + tid; j < end; j += kSlThreads) {
      int32_t e = -1;
      if (held >= 0) {
        if (j < owned) {
          e = old[j];
        } else if (j < owned + got) {
          e = a.ring[ring_at(from + static_cast<long long>(j - owned))];
          if (e < 0 || e >= a.num_pages) bad |= ERR_BAD_PAGE;
        }
      }
      to[j] = e;
    }
  }

  // ---- rows (from the last CTA on: the first ones have one table more) ----
  for (long long r0 = static_cast<long long>(gridDim.x - 1 - blockIdx.x) * kSlThreads; r0 < a.rows;
       r0 += static_cast<long long>(gridDim.x) * kSlThreads) {
    if (a.parents) {
      __syncthreads();  // the block before this one has been walked
      for (int i = tid; i < 2 * kSlTree; i += kSlThreads) {
        const long long r = r0 - kSlTree + i;
        s_parent[i] = r >= 0 && r < a.rows ? a.parents[r] : -1;
      }
      __syncthreads();
    }
    const long long r = r0 + tid;
    if (r >= a.rows) continue;
    int s = 0;  // the last request whose first row is at r or before
    for (int step = a.requests ? 1 << (31 - __clz(a.requests)) : 0; step > 0; step >>= 1)
      if (s + step < a.requests && s_row[s + step] <= r) s += step;
    const int begin = s_row[s], i = static_cast<int>(r) - begin;
    bool ok = r < s_row[a.requests] && !(s_at[s] >> 31);
    int depth = i;
    uint32_t m[kSlTree / 32];
#pragma unroll
    for (int w = 0; w < kSlTree / 32; ++w) m[w] = 0;
    if (ok && a.parents) {
      depth = 0;
      for (int j = i;; ++depth) {  // j falls with every turn
#pragma unroll
        for (int w = 0; w < kSlTree / 32; ++w)
          if (j >> 5 == w) m[w] |= 1u << (j & 31);
        if (j == 0) break;
        const int p = s_parent[kSlTree + tid - i + j];
        if (p < 0 || p >= j) {
          ok = false;
          bad |= ERR_BAD_TREE;
          break;
        }
        j = p;
      }
    } else if (ok && a.mask) {
#pragma unroll
      for (int w = 0; w < kSlTree / 32; ++w) {
        const int k = i + 1 - 32 * w;
        m[w] = k >= 32 ? 0xffffffffu : k > 0 ? (1u << k) - 1u : 0u;
      }
    }
    if (a.seq) a.seq[r] = ok ? s : -1;
    const int held = ok ? a.held[s] : 0;
    if (a.pos) a.pos[r] = ok ? a.base_pos + held + depth : -1;
    if (a.slots) {
      long long slot = -1;
      if (ok) {
        const long long idx = static_cast<long long>(held) + i;
        const int j = static_cast<int>(idx >> a.shift), owned = owned_of(s);
        const int32_t e = j < owned ? a.table[static_cast<long long>(s) * a.width + j]
                                    : a.ring[ring_at((s_at[s] & 0x7fffffffu) + static_cast<long long>(j - owned))];
        if (e >= 0 && e < a.num_pages)
          slot = (static_cast<long long>(e) << a.shift) + (idx & ((1 << a.shift) - 1));
        else
          bad |= ERR_BAD_PAGE;
      }
      a.slots[r] = slot;
    }
    if (a.mask) {
#pragma unroll
      for (int w = 0; w < kSlTree / 32; ++w)
        if (w < a.words) a.mask[r * a.words + w] = ok ? m[w] : 0u;
    }
  }
  if (bad) atomicOr(a.err, bad);
}

}  // namespace
}  // namespace wsg

using namespace wsg;

extern "C" dec_status step_slots(const step_slots_args* a, void* stream) {
  if (!a) return fail(nullptr, DEC_EINVAL, "step_slots: NULL arguments");
  const int shift = page_shift(a->page_size);
  if (a->requests < 0 || a->requests > kSlRequests || a->rows < 0 || a->num_pages < 0 || shift < 0 ||
      a->table_stride < 0 || a->base_pos < 0 || a->mask_words < 0 || a->mask_words > kSlTree / 32 ||
      static_cast<long long>(a->table_stride) << shift > 1ll << 30 || a->base_pos > 1 << 30)
    return fail(nullptr, DEC_EINVAL,
                "step_slots: requests %d, rows %d, num_pages %d, page_size %d, table_stride %d, base_pos %d, mask_words %d",
                a->requests, a->rows, a->num_pages, a->page_size, a->table_stride, a->base_pos, a->mask_words);
  const bool none = a->requests == 0, table = !none && a->table_stride > 0;
  if (!a->free_state || !a->new_free_state || !a->row_start || (a->num_pages > 0 && !a->free_ring) ||
      (!none && (!a->held || !a->fresh || !a->owned || !a->new_owned || !a->ctx_len)) ||
      (table && (!a->page_table || !a->new_table)))
    return fail(nullptr, DEC_EINVAL, "step_slots: NULL pointer");
  if (a->mask && a->mask_words == 0) return fail(nullptr, DEC_EINVAL, "step_slots: a mask of 0 words");
  if (!aligned_to(4, a->held, a->fresh, a->owned, a->parents, a->page_table, a->free_ring, a->free_state, a->new_table,
                  a->new_owned, a->new_free_state, a->row_start, a->ctx_len, a->seq, a->positions, a->mask) ||
      !aligned_to(8, a->slots))
    return fail(nullptr, DEC_EINVAL, "step_slots: a pointer is not aligned to its elements");
  const size_t n = a->requests, r = a->rows, entries = n * a->table_stride;
  const bool in_place = table && a->new_table == a->page_table;
  const Span ring{a->free_ring, 4 * static_cast<size_t>(a->num_pages)};
  const Span row_out[] = {{a->seq, 4 * r}, {a->positions, 4 * r}, {a->slots, 8 * r}, {a->mask, 4 * r * a->mask_words}};
  const std::initializer_list<Span> ins = {{a->held, 4 * n},      {a->fresh, 4 * n}, {a->owned, 4 * n}, {a->parents, 4 * r},
                                           {a->free_state, 8},    {in_place ? nullptr : a->page_table, 4 * entries}};
  if (outputs_meet({ring, {a->new_table, 4 * entries}, {a->new_owned, 4 * n}, {a->new_free_state, 8},
                    {a->row_start, 4 * (n + 1)}, {a->ctx_len, 4 * n}, row_out[0], row_out[1], row_out[2], row_out[3]},
                   ins))
    return fail(nullptr, DEC_EINVAL, "step_slots: an output overlaps another argument");
  DeviceInfo di;
  const dec_status st = device_info(&di, nullptr);
  if (st != DEC_OK) return st;
  SlArgs k{};
  k.requests = a->requests;
  k.rows = a->rows;
  k.num_pages = a->num_pages;
  k.shift = shift;
  k.width = a->table_stride;
  k.base_pos = a->base_pos;
  k.words = a->mask_words;
  k.tree_max = a->mask ? 32 * a->mask_words : a->parents ? kSlTree : 0x7fffffff;
  k.held = a->held;
  k.fresh = a->fresh;
  k.owned = a->owned;
  k.parents = a->parents;
  k.table = a->page_table;
  k.ring = a->free_ring;
  k.state = a->free_state;
  k.new_table = a->new_table;
  k.new_owned = a->new_owned;
  k.new_state = a->new_free_state;
  k.row_start = a->row_start;
  k.ctx_len = a->ctx_len;
  k.seq = a->seq;
  k.pos = a->positions;
  k.slots = a->slots;
  k.mask = a->mask;
  k.in_place = in_place;
  k.err = di.err;
  // a CTA for 256 rows or 1024 table entries, whatever asks for more (2048: 8.6 us for the
  // 256 requests above, 512: 7.8)
  const long long most = di.sms, rows = (r + kSlThreads - 1) / kSlThreads, copies = (entries + 1023) / 1024;
  long long grid = rows > copies ? rows : copies;
  grid = grid < 1 ? 1 : grid > most ? most : grid;
  const size_t smem = 4 * (2 * n + 1);
  WSG_CUDA_TRY(nullptr, launch_k(step_slots_kernel, dim3(static_cast<unsigned>(grid)), dim3(kSlThreads), smem,
                                 static_cast<cudaStream_t>(stream), true, k));
  return DEC_OK;
}
