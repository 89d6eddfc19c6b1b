// kv_layout.cuh -- where each byte of the quantised key/value cache lies
// (include/qmm.h, "Quantised key/value cache"), shared by the kernels that
// write it, read it back and attend to it.
//
// The cache is pages of `page` tokens; a page holds, for each key/value head,
// page / 16 groups of 16 tokens, and a group its key codes, key scales, value
// codes and value scales, one contiguous run of bytes whose length is a
// multiple of 16: one bulk copy brings a group, or several that follow each
// other in a page. Inside a group the codes stand in the order in which the
// lanes of a warp feed them to mma.m16n8k16 (lane = 4 g + t, g < 8, t < 4):
//
//  * keys are the columns of the first product. Column n of the group's half j
//    is token (n >> 1) + 4 (n & 1) + 8 j, and lane (g, t) of column g needs
//    dims 4t .. 4t+3 and 16+4t .. 16+4t+3 of every block, so these bytes stand
//    together for as many blocks as fill 16 bytes (4 of Q4_0, 2 of Q8_0) and
//    the chunks of the 32 lanes follow each other: 128-bit loads without a
//    bank conflict;
//  * values are the columns of the second product, so lane (g, t) needs dims
//    2g, 2g+1, 16+2g and 17+2g of every block of tokens t, t+4, t+8, t+12:
//    8-byte chunks for 4 (2) blocks, and the chunks that 16 lanes load
//    together follow each other;
//  * a scale of each of the four tokens t, t+4, t+8, t+12 is 8 bytes together,
//    for every block of t.
//
// A head size whose block count is not a multiple of 4 (2) is laid out in runs
// of 4 (2), then 2, then 1 blocks.
#pragma once

#include <stdint.h>

namespace qmm {

constexpr int kKvGroup = 16;  // tokens of a group

// Bytes of the keys' (or the values') part of a group: codes, then scales.
__host__ __device__ constexpr int kv_code_bytes(int nb, bool q8) { return nb * (q8 ? 512 : 256); }
__host__ __device__ constexpr int kv_part_bytes(int nb, bool q8) { return kv_code_bytes(nb, q8) + nb * 32; }

// The runs of blocks of a row: how many, a run's first block and its blocks. Plain
// arithmetic on the run's number, which unrolled loops fold: a loop that steps by
// a run's length is not unrolled, and arrays indexed in it lie in local memory
// (attention over 16 x 8192 tokens of 8 heads of 256, Q8_0: 268 us, with this 110).
__host__ __device__ constexpr int kv_runs(int nb, bool q8) { return q8 ? nb / 2 + nb % 2 : nb / 4 + nb % 4 / 2 + nb % 2; }
__host__ __device__ constexpr int kv_run_first(int nb, bool q8, int i) {
  return q8 ? 2 * i : nb % 4 == 3 && i == nb / 4 + 1 ? nb - 1 : 4 * i;
}
__host__ __device__ constexpr int kv_run_blocks(int nb, bool q8, int i) {
  const int left = nb - kv_run_first(nb, q8, i);
  return !q8 && left >= 4 ? 4 : left >= 2 ? 2 : 1;
}

// Byte offset in the part of the fp16 scale of block b of token tok.
__host__ __device__ constexpr int kv_scale_at(int nb, bool q8, int tok, int b) {
  return kv_code_bytes(nb, q8) + ((tok & 3) * nb + b) * 8 + (tok >> 2) * 2;
}

// A cache's form, as the kernels use it.
struct KvForm {
  int nb;            // blocks of a row: head size / 32
  int heads;         // key/value heads
  int page;          // tokens of a page (a power of two, 16 at least)
  bool kq8, vq8;     // Q8_0 (else Q4_0)
  int64_t pages;
  __host__ __device__ int group_bytes() const { return kv_part_bytes(nb, kq8) + kv_part_bytes(nb, vq8); }
  // Offset of group `grp` (of page * heads * groups order) in the cache.
  __host__ __device__ int64_t group_at(int64_t pg, int head, int grp) const {
    return ((pg * heads + head) * (page / kKvGroup) + grp) * static_cast<int64_t>(group_bytes());
  }
};

}  // namespace qmm
