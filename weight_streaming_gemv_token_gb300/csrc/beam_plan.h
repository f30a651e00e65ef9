// How a selection is cut up, where its lists lie and which places of them a thread
// visits: plain C++, so that it can be tested without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>

#if defined(__CUDACC__)
#define WSG_DEV __device__ __forceinline__
#else
#define WSG_DEV inline
#endif

namespace wsg {

constexpr int kBeamThreads = 512;     // of a CTA of pass 2
constexpr int kBeamChunksMax = 4096;  // chunks of one call (all rows)
constexpr int kBeamChunkMin = 128, kBeamChunkUsual = 1024;
constexpr int kBeamGather = 4096;  // candidates held in shared memory

// Workspace: the chunks' maxima with their sums and indices; the arrival counter; per
// qualified chunk a count and a list of (key, flat index).
struct BeamLayout {
  int chunk, per_row, chunks, slots;
  int list;  // places of a slot's list
  size_t part, counter, count, key, flat, total;
};

inline BeamLayout beam_layout(int beams, int vocab, int n_out) {
  BeamLayout L{};
  // The smallest power of two within the bound on the number of chunks, 2,048 for few
  // outputs (every CTA of pass 2 looks at each). Smaller chunks where they are fewer
  // than four times the outputs: the n_out-th best chunk would bound little (4 beams
  // x 151,936, 1,024 outputs: 1,330 us with chunks of 1,024, 91 with 256; 8 outputs: 12).
  const int most = n_out > 256 ? kBeamChunksMax : kBeamChunksMax / 2;
  auto chunks = [&](long long size) { return beams * ((vocab + size - 1) / size); };
  long long c = kBeamChunkUsual;
  while (chunks(c) > most) c *= 2;
  while (c > kBeamChunkMin && chunks(c) < 4ll * n_out && chunks(c / 2) <= most) c /= 2;
  L.chunk = static_cast<int>(c);
  L.per_row = static_cast<int>((vocab + c - 1) / c);
  L.chunks = L.per_row * beams;
  L.slots = n_out < L.chunks ? n_out : L.chunks;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  L.part = take(16 * static_cast<size_t>(L.chunks));
  L.counter = take(4);
  L.count = take(4 * static_cast<size_t>(L.slots));
  L.list = static_cast<int>(c < vocab ? c : vocab);
  const size_t places = static_cast<size_t>(L.slots) * L.list;
  L.key = take(8 * places);
  L.flat = take(4 * places);
  L.total = o;
  return L;
}

// The places that thread `tid` of kBeamThreads visits in lists of `list` places each,
// of which the first count(slot) hold a candidate: w = load(place) of up to eight
// together, then fn(w, place). Behind a list's count nothing is loaded and fn gets a
// word of 0, with which it must return before it touches the place: the end of the last
// list is the end of the workspace. (With a test of the word before fn, 4 beams of equal
// logits, 64 outputs, take 550 us; like this 500.)
template <typename Count, typename Load, typename Fn>
WSG_DEV void beam_walk(int slots, int list, int tid, Count count, Load load, Fn fn) {
  int per = 1;  // threads a list
  while (per < 32 && slots * per * 2 <= kBeamThreads) per *= 2;
#pragma unroll 1
  for (int q = tid / per; q < slots; q += kBeamThreads / per) {
    const uint32_t n = count(q);
    const size_t p0 = static_cast<size_t>(q) * list;
#pragma unroll 1
    for (uint32_t i0 = tid & (per - 1); i0 < n; i0 += 8 * per) {
      uint32_t k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        k[e] = i0 + e * per < n ? load(p0 + i0 + e * per) : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        fn(k[e], p0 + i0 + e * per);
    }
  }
}

}  // namespace wsg
