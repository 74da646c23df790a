// Where the persistent prompt kernels (prefill_packed.cu, prefill_int8.cu) find their
// work: lengths are on the device only, so a warp of each CTA looks for its items.
//
// An item is a span of a sequence's tokens and a kv head. Items are ranked by level (the
// span's place in its sequence) from the highest down, then by sequence, then by kv head;
// CTA c of N takes ranks c, 2 N - 1 - c, 2 N + c ... Ranks only go up, so a place in that
// order moves along: 32 sequences at a time (a batch, one a lane), then the next level.
//
// One long prompt among thousands of short ones has many levels that few sequences
// reach. So the place passes only over batches that have one (runs of batches whose
// longest is known, one run a lane: up to 1024 sequences a run is a batch), and where an
// item is far, levels that the same sequences reach are passed by a division: 8192 tokens
// (128 levels) among 4000 prompts of one token, 4 heads of 64: 199 us packed and 246 over
// an INT8 cache (the parts alone 172 and 220), by every batch of every level 2890 and
// 3170. Batches that are all alike pay for it: 1024 prompts of 32 tokens, 32/8 heads of
// 128, 199 us where plain counting up takes 195; 256 of 64 to 2048, 721 and 712.
#pragma once

#include <cstdint>

namespace pd {

// Counts: load(sequence) reads what tokens(that, whether to tell of counts that do not
// fit) makes a number of tokens of; a Counts::Raw of zeros means none. Apart, so that the
// counts of the batch to come are on their way while this one's items are worked on.
template <class Counts>
struct ItemSearch {
  using Raw = typename Counts::Raw;
  struct Found {
    int b, n, tok0, g;  // tok0: the span's first token; g = -1: no items left
  };
  Counts counts;
  int lane, num_seqs, span, hkv;
  // What only the ends of levels need, a word a lane each: the run's longest sequence's
  // tokens; the pairs before the level
  int* longest;
  int* start;
  uint32_t live;        // the runs with a sequence that reaches the level
  int edge;             // the level: its spans' first token (negative: no level left)
  int batch, before;    // the place: a batch, and the (sequence, level) pairs before it
  int now;              // tokens of the lane's sequence in the batch
  int ahead_at;         // the batch to come (not past this one: the next level's first)
  Raw ahead;            // and the counts of the lane's sequence in that
  int round;

  __device__ __forceinline__ int batches() const { return (num_seqs + 31) >> 5; }
  __device__ __forceinline__ int per_run() const { return (num_seqs + 1023) >> 10; }
  __device__ __forceinline__ Raw raw_at(int batch) const {
    const int b = batch * 32 + lane;
    return b < num_seqs ? counts.load(b) : Raw{};
  }
  __device__ __forceinline__ int tokens_at(int batch, bool tell) const {
    return counts.tokens(raw_at(batch), tell);
  }
  __device__ __forceinline__ int most_of(int n) const {
    return __reduce_max_sync(0xFFFFFFFFu, n);
  }
  __device__ __forceinline__ uint32_t live_runs() const {
    return __ballot_sync(0xFFFFFFFFu, *longest > edge);
  }
  __device__ __forceinline__ int first_live() const { return (__ffs(live) - 1) * per_run(); }
  // The batch of a live run behind `at`, or the first one.
  __device__ __forceinline__ int behind(int at) const {
    int run = at;
    if (per_run() > 1) {
      if (at + 1 >= batches()) return first_live();
      run = at / per_run();
      if ((at + 1) / per_run() == run) return at + 1;
    }
    const uint32_t rest = (live >> run) >> 1;
    return rest ? (run + __ffs(rest)) * per_run() : first_live();
  }
  __device__ __forceinline__ void look_ahead() {
    ahead_at = behind(batch);
    ahead = raw_at(ahead_at);
  }
  __device__ __forceinline__ void go_to_first() {
    live = live_runs();
    *start = before;
    batch = first_live();
    now = tokens_at(batch, false);
    look_ahead();
  }
  // From the start of a level that `count` sequences reach, past the levels that the same
  // ones reach and behind which the pair pr lies. most: tokens of the longest other one.
  __device__ __forceinline__ void leap(int pr, int count, int most) {
    if (count == 0) {  // not while the lengths stay as they are
      edge = -1;
      return;
    }
    const int skip = min((pr - before) / count, (edge - most) / span + 1);
    before += skip * count;
    edge -= skip * span;
  }
  __device__ __forceinline__ void leap_batches(int pr) {
    live = live_runs();
    int most = *longest > edge ? 0 : *longest, count = 0;
    int i = first_live(), last;
    do {
      const int n = tokens_at(i, false);
      count += __popc(__ballot_sync(0xFFFFFFFFu, n > edge));
      if (n <= edge) most = max(most, n);
      last = i;
      i = behind(i);
    } while (i > last);
    leap(pr, count, most_of(most));
  }
  __device__ __forceinline__ ItemSearch(const Counts& c, int lane, int num_seqs, int span, int hkv,
                                        bool tell, int (*words)[32])
      : counts(c), lane(lane), num_seqs(num_seqs), span(span), hkv(hkv) {
    round = before = batch = ahead_at = 0;
    ahead = Raw{};
    longest = &words[0][lane];
    start = &words[1][lane];
    *longest = 0;
    live = 1u;
    int top = 0;
    if (batches() <= 1) {
      now = tokens_at(0, tell);
      top = most_of(now);
    } else {
      for (int i = 0, run = 0; i < batches(); ++run) {
        int most = 0;
        for (const int end = min(i + per_run(), batches()); i < end; ++i)
          most = max(most, tokens_at(i, tell));
        most = most_of(most);
        if (run == lane) *longest = most;
        top = max(top, most);
      }
    }
    edge = (top + span - 1) / span * span - span;
    if (batches() > 1) {  // behind a level of none, which the first search leaves
      now = 0;
      edge += span;
      *start = 0;
    }
  }
  // This CTA's next item.
  __device__ __forceinline__ Found next() {
    Found it = {0, 0, 0, -1};
    const int64_t rank = static_cast<int64_t>(round) * gridDim.x +
                         ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    ++round;
    const int64_t pr64 = rank <= UINT32_MAX
                             ? static_cast<uint32_t>(rank) / static_cast<uint32_t>(hkv)
                             : rank / hkv;
    if (pr64 > INT32_MAX) return it;
    const int pr = static_cast<int>(pr64);  // the (sequence, level) pair
    while (edge >= 0) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, now > edge);
      const int c = __popc(m);
      if (pr - before < c) {
        uint32_t left = m;
        for (int i = before; i < pr; ++i) left &= left - 1;
        const int src = __ffs(left) - 1;
        it.n = __shfl_sync(0xFFFFFFFFu, now, src);
        it.b = batch * 32 + src;
        it.tok0 = edge;
        it.g = static_cast<int>(rank - pr64 * hkv);
        break;
      }
      if (batches() == 1) {
        // a leap from eight levels' worth on (one prompt of 4096 tokens, 64 levels,
        // head_dim 256: 57.7 us, level by level 60.6)
        if (pr - before >= 8 * c) {
          leap(pr, c, most_of(now > edge ? 0 : now));
        } else {
          before += c;
          edge -= span;
        }
        continue;
      }
      before += c;
      if (ahead_at > batch) {
        batch = ahead_at;
        now = counts.tokens(ahead, false);
        look_ahead();
        continue;
      }
      // the level's end
      const int passed = before - *start;
      edge -= span;
      if (edge >= 0 && passed > 0 && pr - before >= 8 * passed) leap_batches(pr);
      if (edge >= 0) go_to_first();
    }
    return it;
  }
};

}  // namespace pd
