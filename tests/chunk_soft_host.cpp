// The softmax warps of the tcgen05 chunk kernels on the CPU: soft_warp of csrc/vq_chunk_soft.cuh, as the
// kernel runs it, over eight simulated warps whose waits give up at random moments, each for itself.
// One warp runs at a time; who goes on is drawn.  A schedule in which nobody can go on is a hang.
//
//   chunk_soft_host <schedules> <leave>     leave 1: a warp that gave up leaves at once instead
// prints: schedules that hung, schedules in which a warp gave up, schedules in which one warp of a row gave
// up at a wait that the other passed, schedules that came to their end with every piece stored.
#include <ucontext.h>

#include <cstdio>
#include <cstdlib>
#include <functional>
#include <random>
#include <vector>

#include "../bit_vector_quantized_gb300/csrc/vq_chunk_soft.cuh"

namespace {

constexpr int kWarps = 8;

// The order before: a warp leaves its loops where a wait gave up.
template <typename Take, typename LoadQuery, typename AllTook, typename TurnHalf, typename RowSync, typename Turn,
          typename ScoresWait, typename BlockHalf, typename Block, typename OutputWait, typename PutSum, typename Store>
void leaving_warp(Take take, LoadQuery, AllTook all_took, TurnHalf, RowSync row_sync, Turn turn, ScoresWait scores_wait,
                  BlockHalf, Block block, OutputWait output_wait, PutSum, Store store) {
  while (take()) {
    all_took(true);
    row_sync();
    const int blocks = turn();
    for (int j = 0; j < blocks; ++j) {
      if (!scores_wait()) return;
      row_sync();
      if (!block(j, blocks)) return;
    }
    if (!output_wait(blocks)) return;
    row_sync();
    store();
    row_sync();
  }
}

struct Barrier {
  int need, here = 0, round = 0;
};

struct Sim {
  std::mt19937 rng;
  bool leave, late = false, abort_flag = false;
  std::vector<int> pieces;  // blocks of each
  Barrier rows[kWarps / 2], all;
  std::vector<int> arrived;  // by block over all pieces: warps whose P is there
  std::vector<int> queried;  // by piece: warps whose Q~ is there
  int stores = 0, blocks_total = 0;
  std::vector<std::vector<int>> outcome;  // [warp] of its waits, in order
  ucontext_t main, ctx[kWarps];
  std::vector<std::vector<char>> stacks;
  std::function<bool()> until[kWarps];
  bool done[kWarps] = {};
  int me = 0;

  explicit Sim(unsigned seed, bool leave_) : rng(seed), leave(leave_) {
    for (int n = 1 + rng() % 3; n > 0; --n) {
      pieces.push_back(1 + rng() % 4);
      blocks_total += pieces.back();
    }
    for (auto& r : rows) r.need = 2;
    all.need = kWarps;
    arrived.assign(blocks_total, 0);
    queried.assign(pieces.size(), 0);
    outcome.resize(kWarps);
    stacks.resize(kWarps, std::vector<char>(1 << 16));
  }
  void block_until(std::function<bool()> f) {
    until[me] = std::move(f);
    swapcontext(&ctx[me], &main);
  }
  void meet(Barrier& b) {
    const int round = b.round;
    if (++b.here == b.need) {
      b.here = 0;
      ++b.round;
    }
    block_until([&b, round] { return b.round != round; });
  }
  // A bounded wait: the phase first, then the flag, then the time, as the kernel's.
  bool wait(std::function<bool()> complete) {
    block_until([this, complete] { return complete() || abort_flag || late; });
    const bool ok = complete();
    if (!ok) abort_flag = true;
    outcome[me].push_back(ok);
    return ok;
  }
  void warp() {
    const int w = me;
    unsigned piece = 0;
    int first = 0, j_now = 0;  // blocks before this piece, and of it
    auto take = [&] {
      const bool there = wait([&, this] { return true; });
      return there && piece < pieces.size();
    };
    auto load_query = [] {};
    auto all_took = [&](bool took) {
      const size_t at = vote_at[w]++;
      if (votes.size() <= at) votes.resize(at + 1, 1);
      if (!took) votes[at] = 0;
      meet(all);
      return votes[at] != 0;
    };
    auto turn_half = [] {};
    auto row_sync = [&] { meet(rows[w & 3]); };
    auto turn = [&] {
      ++queried[piece];
      j_now = 0;
      return pieces[piece];
    };
    auto scores = [&](int j) {  // scores of block j of the piece: Q~ of all, and P of block j - 2
      return queried[piece] == kWarps && (j < 2 || arrived[first + j - 2] == kWarps);
    };
    auto scores_wait = [&] { return wait([&, this] { return scores(j_now); }); };
    auto block_half = [](int) {};
    auto block = [&](int j, int blocks) {
      if (j > 0 && rng() % 4 == 0 && !wait([&, this] { return j + 1 < blocks ? scores(j + 1) : arrived[first + j - 1] == kWarps; }))
        return false;
      ++arrived[first + j];
      ++j_now;
      return true;
    };
    auto output_wait = [&](int blocks) { return wait([&, this] { return arrived[first + blocks - 1] == kWarps; }); };
    auto put_sum = [] {};
    auto store = [&] {
      ++stores;
      first += pieces[piece++];
    };
    if (leave) leaving_warp(take, load_query, all_took, turn_half, row_sync, turn, scores_wait, block_half, block, output_wait, put_sum, store);
    else vqk::soft_warp(take, load_query, all_took, turn_half, row_sync, turn, scores_wait, block_half, block, output_wait, put_sum, store);
    done[w] = true;
    swapcontext(&ctx[w], &main);
  }
  std::vector<char> votes;
  size_t vote_at[kWarps] = {};

  static Sim* current;
  static void entry() { current->warp(); }
  // false: nobody can go on
  bool run() {
    current = this;
    const unsigned limit = rng() % 3 ? rng() % (40 * blocks_total) : ~0u;  // when the waits' time is gone
    for (me = 0; me < kWarps; ++me) {
      getcontext(&ctx[me]);
      ctx[me].uc_stack.ss_sp = stacks[me].data();
      ctx[me].uc_stack.ss_size = stacks[me].size();
      ctx[me].uc_link = &main;
      makecontext(&ctx[me], entry, 0);
      until[me] = [] { return true; };
    }
    for (unsigned step = 0;; ++step) {
      if (step >= limit) late = true;
      std::vector<int> ready;
      bool open = false;
      for (int w = 0; w < kWarps; ++w)
        if (!done[w]) {
          open = true;
          if (until[w]()) ready.push_back(w);
        }
      if (!open) return true;
      if (ready.empty()) return false;
      me = ready[rng() % ready.size()];
      swapcontext(&main, &ctx[me]);
    }
  }
};
Sim* Sim::current = nullptr;

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  int hung = 0, gave_up = 0, split = 0, whole = 0;
  for (int seed = 0; seed < std::atoi(argv[1]); ++seed) {
    Sim s(seed, std::atoi(argv[2]) != 0);
    if (!s.run()) ++hung;
    bool any = false, differ = false;
    for (int w = 0; w < kWarps; ++w)
      for (size_t i = 0; i < s.outcome[w].size(); ++i)
        if (!s.outcome[w][i]) {
          any = true;
          const auto& o = s.outcome[w ^ 4];
          differ = differ || (i < o.size() && o[i]);
        }
    gave_up += any;
    split += differ;
    whole += !any && s.stores == kWarps * static_cast<int>(s.pieces.size());
  }
  std::printf("%d %d %d %d\n", hung, gave_up, split, whole);
}
