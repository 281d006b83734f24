// The rings' sizes as the kernels have them, and the plan of tree attention (csrc/vq_chunk_plan.cuh with kTree) run on the
// host: worker and blocks of every piece.
#include "../bit_vector_quantized_gb300/csrc/vq_chunk_plan.cuh"

extern "C" int ring_slots(int tree) { return tree ? vqk::kTreePieces : vqk::kWidePieces; }

extern "C" long long ring_blocks(int tile_tok, int gap, int hkv, int batch, const int* lens, const int* cu, int workers, int max_seq_len,
                                 int* out, long long cap) {
  vqk::ChunkParams p{};
  p.seq_lens = lens;
  p.cu = cu;
  p.batch = batch;
  p.hkv = hkv;
  p.num_tokens = cu[batch];
  p.max_seq_len = max_seq_len;
  p.max_new_len = 256;
  p.tile_tok = tile_tok;
  p.gap = gap;
  p.min_range = 512;
  static long long pre[vqk::kChunkMaxBatch + 1];
  pre[0] = 0;
  for (int b = 0; b < batch; ++b) {  // (tree_plan's sums)
    const vqk::ChunkSeq s = vqk::chunk_seq<true>(p, b);
    pre[b + 1] = pre[b] + p.hkv * vqk::chunk_sum<true>(p, s, (s.n + tile_tok - 1) / tile_tok);
  }
  long long n = 0;
  for (int me = 0; me < workers; ++me) {
    vqk::ChunkWalk<128, true> walk;
    walk.start(p, pre, me, workers);
    vqk::ChunkPiece q;
    while (walk.next(p, q)) {
      if (n < cap) {
        out[2 * n] = me;
        out[2 * n + 1] = q.blk1 - q.blk0;
      }
      ++n;
    }
  }
  return n;
}
