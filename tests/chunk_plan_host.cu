// The plan of the chunk-attention kernels (csrc/vq_chunk_plan.cuh), run on the host: every piece of every worker.
#include "../bit_vector_quantized_gb300/csrc/vq_chunk_plan.cuh"

namespace {

template <int CW>
long long pieces(const vqk::ChunkParams& p, int workers, int* out, long long cap) {
  static long long pre[vqk::kChunkMaxBatch + 1];
  pre[0] = 0;
  for (int b = 0; b < p.batch; ++b) {  // (chunk_plan's sums)
    const vqk::ChunkSeq s = vqk::chunk_seq(p, b);
    pre[b + 1] = pre[b] + p.hkv * vqk::chunk_sum(p, s, (s.n + p.tile_tok - 1) / p.tile_tok);
  }
  long long n = 0;
  for (int me = 0; me < workers; ++me) {
    vqk::ChunkWalk<CW> walk;
    walk.start(p, pre, me, workers);
    vqk::ChunkPiece q;
    while (walk.next(p, q)) {
      if (n < cap) {
        const int row[] = {me, q.b, q.kvh, q.tile, q.blk0, q.blk1, q.slot, q.last, q.k.sink, q.k.lo, q.k.count};
        for (int i = 0; i < 11; ++i) out[11 * n + i] = row[i];
      }
      ++n;
    }
  }
  return n;
}

}  // namespace

extern "C" long long chunk_plan_pieces(int block, int tile_tok, int gap, int min_range, int window, int sinks, int hkv,
                                       int batch, const int* lens, const int* cu, int max_seq_len, int max_new_len,
                                       int num_tokens, int workers, int* out, long long cap) {
  vqk::ChunkParams p{};
  p.seq_lens = lens;
  p.cu = cu;
  p.batch = batch;
  p.hkv = hkv;
  p.num_tokens = num_tokens;
  p.max_seq_len = max_seq_len;
  p.max_new_len = max_new_len;
  p.window = window;
  p.sinks = sinks;
  p.tile_tok = tile_tok;
  p.gap = gap;
  p.min_range = min_range;
  return block == 16 ? pieces<16>(p, workers, out, cap) : pieces<128>(p, workers, out, cap);
}
