// How a call of attn_shared_prefix is cut up, and its limits on sizes: host
// arithmetic in plain C++, so that it can be tested without a GPU.
#pragma once
#include <cmath>
#include <cstdint>

#include "../../include/wsg.h"
#include "paging.h"

namespace wsg {

constexpr int kAmWarps = 8;                               // warps of attn_f32_kernel's CTAs
constexpr int kApD = 128, kApRows = 128, kApKeys = 128;  // attn_prefix_tc_kernel: head size, rows a CTA, keys a tile

inline bool attn_sizes_ok(const attn_shared_args* a) {
  auto type = [](int t) { return t == DEC_F32 || t == DEC_BF16; };
  return a->batch >= 0 && a->batch <= 65535 && a->n_kv >= 1 && a->n_q >= a->n_kv && a->n_q <= 65535 &&
         static_cast<long long>(a->batch) * a->n_q < 1ll << 24 &&
         a->n_q % a->n_kv == 0 && a->n_q / a->n_kv <= 16 && a->head_dim >= 8 && a->head_dim <= 128 &&
         a->head_dim % 8 == 0 && type(a->qdtype) && type(a->kvdtype) && a->prefix_len >= 0 &&
         page_shift(a->page_size) >= 0 && a->num_pages >= 0 && a->table_stride >= 0 &&
         (static_cast<long long>(a->table_stride) << page_shift(a->page_size)) + a->prefix_len <= (1ll << 30);
}

// How a call is cut up.
struct AsPlan {
  bool tc;  // the prefix on attn_prefix_tc_kernel (row_groups: blocks of 128 rows)
  bool own_joins;  // ... and the own keys on attn_own_kernel, which joins
  int na, row_groups;  // rows of a prefix item otherwise (0 with tc)
  int prefix_slots, prefix_chunk, own_slots, own_block;
  long long own_seg, own_per;
  long long prefix_items, own_items;  // CTAs
  size_t o, ml, total;                // workspace offsets and size
};

inline AsPlan attn_plan(const attn_shared_args* a, int sms) {
  AsPlan p{};
  p.total = 256;
  if (a->batch == 0) return p;  // an empty call: nothing to share out
  auto up = [](long long x, long long y) { return (x + y - 1) / y; };
  auto least = [](long long x, long long y) { return x < y ? x : y; };
  auto root = [](long long x) { return static_cast<long long>(std::sqrt(static_cast<double>(x))); };
  const bool f32 = a->kvdtype == DEC_F32;
  const int group = a->n_q / a->n_kv, rows = a->batch * group;
  // Queries and cache in bfloat16, head size 128: the prefix on tcgen05 for any number
  // of rows (12 rows x 4096 keys: 9.1 us, with attn_rows_kernel 11.7; 8 rows: the same).
  const bool fast = !f32 && a->qdtype == DEC_BF16 && a->head_dim == kApD && a->prefix_stride < 1ll << 31;
  p.tc = fast && a->prefix_len > 0;
  p.na = fast ? 0 : f32 || rows > 8 ? 16 : 8;
  const int block = fast ? kApRows : p.na;
  p.row_groups = static_cast<int>(up(rows, block));
  const long long capacity = static_cast<long long>(a->table_stride) << page_shift(a->page_size);
  const long long segments = static_cast<long long>(a->batch) * a->n_kv;      // of own keys
  const long long heads = static_cast<long long>(a->n_kv) * p.row_groups;     // prefix items of a split
  // an axis of `keys` keys into about `want` splits of whole units
  auto cut = [&](long long keys, long long unit, long long want, int* slots, int* chunk) {
    const long long per = up(up(keys, unit), want < 1 ? 1 : want);
    *chunk = static_cast<int>((per < 1 ? 1 : per) * unit);
    *slots = static_cast<int>(up(keys, *chunk));
  };
  if (f32) {
    // One CTA an SM. The branches' CTAs follow the prefix's and fill its gaps, so
    // the number of splits is the one with the least estimated end: the longer of a
    // prefix CTA and an SM's share of all, half a CTA more where the last wave is
    // ragged, and 0.06 of a unit of keys for each split to join (8 x 3001: 12 splits
    // 17.2 us, 11 in one wave with the branches' 18.5; 64 x 8192: 2 splits 136, 1 216).
    constexpr int unit = kAmWarps * 8;
    const long long units = up(a->prefix_len, unit), own = up(capacity, unit);
    cut(capacity, unit, own ? sms / ((units ? 2 : 1) * segments) : 0, &p.own_slots, &p.own_block);
    const double each = static_cast<double>(p.own_block) / unit, all = each * p.own_slots * segments;
    long long best = 1;
    double least_end = 0;
    for (long long n = 1; n <= units && n <= 128; ++n) {
      const double chunk = static_cast<double>(up(units, n)), share = (chunk * n * heads + all) / sms;
      const double end = (n * heads > sms ? share + 0.5 * chunk : chunk > share + 0.5 * each ? chunk : share + 0.5 * each) + 0.06 * n;
      if (n == 1 || end < least_end) best = n, least_end = end;
    }
    cut(a->prefix_len, unit, best, &p.prefix_slots, &p.prefix_chunk);
    p.own_seg = p.own_slots;
    p.own_per = 1;
    p.own_items = p.own_slots * segments;
  } else {
    p.own_block = 16;
    p.own_seg = up(capacity, 16);
    const long long line = p.own_seg * segments;  // own blocks
    long long warps;                              // that walk it
    if (fast) {
      // A tile takes about 1 us where CTAs are few, a split 0.1 us to join: no more
      // splits than the square root of ten times the tiles.
      cut(a->prefix_len, kApKeys, least(sms / heads, root(10 * up(a->prefix_len, kApKeys))), &p.prefix_slots,
          &p.prefix_chunk);
      // One CTA walks a branch's keys of a head and joins, unless there are few
      // branches and many keys: 17 branches of one head x 512 own keys take 10.1 us
      // with that and 11.2 with equal pieces for all warps and a join kernel, x 1024
      // 15.1 and 11.2; 160 (branch, head) pairs x 1024 23 and 27.
      p.own_joins = p.own_seg <= 32 || segments >= sms;
      // Otherwise: one CTA of four warps fits beside a prefix CTA, three an SM after
      // those have ended; a second wave pays when the first would walk over 8 blocks a warp.
      warps = 4ll * sms;
      if (line > 8 * warps) warps *= 3;
    } else {
      // one CTA of eight warps an SM, shared out by the number of keys
      const long long units = up(a->prefix_len, 128) * heads;
      const long long pre = units ? sms * units / (units + up(line, 8)) : 0;
      cut(a->prefix_len, 64, least(pre / heads, root(10 * up(a->prefix_len, 64))), &p.prefix_slots, &p.prefix_chunk);
      const long long left = sms - p.prefix_slots * heads;
      warps = 8 * (left > sms / 4 ? left : sms / 4);
    }
    p.own_per = line > 0 ? up(line, warps) : 1;
    p.own_items = up(up(line, p.own_per), fast ? 4 : 8);
    p.own_slots = p.own_seg > 0 ? static_cast<int>((p.own_seg - 1 + p.own_per - 1) / p.own_per + 1) : 0;
    if (p.own_joins) p.own_items = segments, p.own_slots = 0;
  }
  p.prefix_items = p.prefix_slots * heads;
  const long long parts = static_cast<long long>(p.prefix_slots + p.own_slots) * a->batch * a->n_q;
  p.o = 0;
  p.ml = (static_cast<size_t>(parts) * a->head_dim * 4 + 255) / 256 * 256;
  p.total = (p.ml + static_cast<size_t>(parts) * 8 + 256) / 256 * 256;
  return p;
}

}  // namespace wsg
