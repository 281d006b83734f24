// vq_chunk_soft.cuh -- in which order a softmax warp of the tcgen05 chunk kernels waits and meets the others.
//
// A wait on an mbarrier may give up, and in one warp alone: a warp that looks
// a moment later may find the phase complete and go on.  The barriers that
// warps share have no limit, so a warp must not leave while another may still
// come to one of them.  Hence
//   * a warp that gave up keeps to its row barriers, without the work between
//     them, until the end of the piece: 3 + blocks of them whatever happens;
//   * whether there is another piece is voted on by all the warps: they take
//     it, or leave, together.
// So every warp meets the same barriers in the same order, and what is left
// of a piece without its work costs no wait.  (Nothing here is CUDA's, so that
// a program on the host can run it with warps of its own.)
#pragma once

namespace vqk {

// take() -> bool: waits for the next piece (false: none, or gave up); all_took(bool) -> bool: meets all
// warps, true if all took it; row_sync(): meets the row's other warp; turn() -> the piece's blocks;
// scores_wait(), output_wait(blocks) -> bool: false where they gave up; block(j, blocks) -> bool: the same
// for its own wait.
template <typename Take, typename LoadQuery, typename AllTook, typename TurnHalf, typename RowSync, typename Turn, typename ScoresWait,
          typename BlockHalf, typename Block, typename OutputWait, typename PutSum, typename Store>
#ifdef __CUDACC__
__host__ __device__ __forceinline__
#endif
void soft_warp(Take take, LoadQuery load_query, AllTook all_took, TurnHalf turn_half, RowSync row_sync, Turn turn, ScoresWait scores_wait,
               BlockHalf block_half, Block block, OutputWait output_wait, PutSum put_sum, Store store) {
  bool ok = true;
  for (;;) {
    ok = ok && take();
    load_query();
    if (!all_took(ok)) return;
    turn_half();
    row_sync();
    const int blocks = turn();
    for (int j = 0; j < blocks; ++j) {
      if (!ok || !scores_wait()) {
        ok = false;
        row_sync();
        continue;
      }
      block_half(j);
      row_sync();
      ok = block(j, blocks);
    }
    if (!ok || !output_wait(blocks)) {
      ok = false;
      row_sync();
      row_sync();
      continue;
    }
    put_sum();
    row_sync();
    store();
    row_sync();  // the row's shared memory is free again
  }
}

}  // namespace vqk
