// Every interleaving of two data warps, the issuing warp and the tensor core of the packed state kernel,
// for chunks of given numbers of steps.  An mbarrier is the number of its completed phases; a wait for
// parity p passes while the phase at work has the other parity.
//   argv: rule (0: a warp waits wherever it wants to know, 1: StepsDone), then steps of each chunk.
// Prints "ok", "stuck" (an interleaving in which nobody can go on) or "early" (a wait passed too soon).
#include <cstdio>
#include <cstdlib>
#include <set>
#include <tuple>
#include <vector>

#include "steps_done.h"

struct Op {
  bool wait;  // for step's products; else arrive: the step's operands are ready
  int step;
};

static std::vector<Op> warp_ops(const std::vector<int>& chunks, bool rule) {
  std::vector<Op> ops;
  retnet::StepsDone steps;
  auto wait = [&](int n) {
    if (rule && !steps.must_wait(n)) return;
    ops.push_back({true, n});
    steps.waited(n);
  };
  int n = 0, last_step = -1;
  for (size_t c = 0; c < chunks.size(); ++c) {
    for (int s = 0; s < chunks[c]; ++s, ++n) {
      if (n >= 2) wait(n - 2);
      ops.push_back({false, n});
    }
    if (c > 0) wait(last_step);
    last_step = n - 1;
  }
  wait(last_step);
  return ops;
}

int main(int argc, char** argv) {
  std::vector<int> chunks;
  int total = 0;
  for (int i = 2; i < argc; ++i) {
    chunks.push_back(std::atoi(argv[i]));
    total += chunks.back();
  }
  const std::vector<Op> ops = warp_ops(chunks, std::atoi(argv[1]) != 0);
  using State = std::tuple<int, int, int, int>;  // places of the two warps, steps issued, steps done
  std::set<State> seen;
  std::vector<State> todo{{0, 0, 0, 0}};
  auto of_parity = [](int steps, int p) { return (steps + 1 - p) / 2; };  // among steps 0 .. steps - 1
  auto arrived = [&](int place, int p) {
    int n = 0;
    for (int i = 0; i < place; ++i) n += !ops[i].wait && (ops[i].step & 1) == p;
    return n;
  };
  const int end = static_cast<int>(ops.size());
  while (!todo.empty()) {
    const State at = todo.back();
    todo.pop_back();
    if (!seen.insert(at).second) continue;
    const auto [a, b, issued, done] = at;
    bool moved = false;
    for (int w = 0; w < 2; ++w) {
      const int place = w ? b : a;
      if (place == end) continue;
      const Op op = ops[place];
      if (op.wait) {
        const int phases = of_parity(done, op.step & 1);
        if ((phases & 1) == ((op.step >> 1) & 1)) continue;
        if (done <= op.step) return std::puts("early"), 0;
      }
      todo.push_back(w ? State{a, b + 1, issued, done} : State{a + 1, b, issued, done});
      moved = true;
    }
    if (issued < total) {  // the issuing warp: waits for the step's operands, then issues
      const int p = issued & 1, phases = (arrived(a, p) + arrived(b, p)) / 2;
      if ((phases & 1) != ((issued >> 1) & 1)) {
        if (phases <= issued / 2) return std::puts("early"), 0;
        todo.push_back({a, b, issued + 1, done});
        moved = true;
      }
    }
    if (done < issued) {
      todo.push_back({a, b, issued, done + 1});
      moved = true;
    }
    if (!moved && (a < end || b < end || done < total)) return std::puts("stuck"), 0;
  }
  std::puts("ok");
}
