// How a CTA of the norm of queries and keys walks over its heads.
#pragma once

#ifdef __CUDACC__
#define MHLA_HEADS_FN __host__ __device__ __forceinline__
#else
#define MHLA_HEADS_FN inline
#endif

namespace mhla {

// Heads first .. last - 1 of a CTA, counted over q's heads and then k's; those from
// `split` on are k's.
struct HeadShare {
  int first, split, last;

  MHLA_HEADS_FN HeadShare(int part, int per, int q_heads, int all) {
    first = part * per;
    last = first + per < all ? first + per : all;
    split = q_heads < first ? first : q_heads > last ? last : q_heads;
  }
  // Behind the last head of the step that begins at `h`: at most `rows` heads, of
  // one tensor, all of them there.
  MHLA_HEADS_FN int step_end(int h, int rows) const {
    const int end = h < split ? split : last;
    return h + rows < end ? h + rows : end;
  }
};

}  // namespace mhla

#undef MHLA_HEADS_FN
