// norm_keep.h - which of the gradient norm's chunks stay in the last-level cache.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ps {

// Index of the first chunk from which on whole chunks are read so that they stay
// in the cache: those of at most `keep` bytes, from the last one on. Parts of a
// chunk are read past the cache and take nothing of it. A tensor that has no
// gradient counts like any other: one may come.
// tensors: what the norm reads, in order; size_of(t): elements, and bytes of each.
template <class V, class F>
uint64_t norm_keep_from(const V& tensors, F size_of, int64_t chunk, int64_t keep) {
  uint64_t from = 0;
  for (const auto& t : tensors) from += (uint64_t)((size_of(t).first + chunk - 1) / chunk);
  for (size_t k = tensors.size(); k-- > 0;) {
    const auto [n, bytes] = size_of(tensors[k]);
    const int64_t whole = n / chunk, part = n % chunk != 0, fit = keep / (chunk * bytes);
    from -= (uint64_t)(part + (whole < fit ? whole : fit));
    if (whole > fit) break;
    keep -= whole * chunk * bytes;
  }
  return from;
}

}  // namespace ps
