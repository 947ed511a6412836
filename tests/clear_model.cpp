// The training kernels' clearing warp (attn_tiles.cuh) on the host: the load thread, the MMA warp and the clearing
// warp as coroutines on model barriers, the clearing warp last of all to be given the processor.  What is under
// test is the header's own code; the other two roles go through a ring of tiles as the kernels do.
// Compiled by test_clear_warp.py with -DSA_RING=<slots> -DSA_FIRST=<0 or 1>.
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <vector>

#include "attn_tiles.cuh"

using namespace sa;
using namespace sa::tiles;

namespace model {
ucontext_t scheduler;
struct Role {
  ucontext_t at;
  std::vector<char> stack = std::vector<char>(1 << 18);
  std::function<void()> body;
  uint64_t* bar = nullptr;   // waited for
  uint32_t parity = 0;
  bool done = false;
};
std::vector<Role*> roles;
Role* running = nullptr;
std::vector<uint4*> asked;   // answers to come

// A barrier's word: phase in the low 32 bits, then 16 bits of arrivals to come and 16 of arrivals a phase.
uint32_t phase(uint64_t w) { return (uint32_t)w; }
uint32_t pending(uint64_t w) { return (uint32_t)(w >> 32) & 0xffffu; }
uint32_t count(uint64_t w) { return (uint32_t)(w >> 48); }
uint64_t word(uint32_t phase, uint32_t pending, uint32_t count) {
  return ((uint64_t)count << 48) | ((uint64_t)pending << 32) | phase;
}
void init(uint64_t* bar, uint32_t n) { *bar = word(0, n, n); }
void arrive(uint64_t* bar) {
  const uint64_t w = *bar;
  *bar = pending(w) == 1 ? word(phase(w) + 1, count(w), count(w)) : word(phase(w), pending(w) - 1, count(w));
}
bool passes(const uint64_t* bar, uint32_t parity) { return (phase(*bar) & 1u) != parity; }
void wait(uint64_t* bar, uint32_t parity) {
  if (passes(bar, parity)) return;
  running->bar = bar;
  running->parity = parity;
  swapcontext(&running->at, &scheduler);
}
void start() {
  running->body();
  running->done = true;
  swapcontext(&running->at, &scheduler);
}
void add(std::function<void()> body) {
  Role* r = new Role;
  r->body = body;
  getcontext(&r->at);
  r->at.uc_stack.ss_sp = r->stack.data();
  r->at.uc_stack.ss_size = r->stack.size();
  makecontext(&r->at, start, 0);
  roles.push_back(r);
}
// The first role that can go on does, until it waits.  False: some wait for ever.
bool run() {
  for (;;) {
    Role* next = nullptr;
    bool left = false;
    for (Role* r : roles) {
      if (r->done) continue;
      left = true;
      if (r->bar == nullptr || passes(r->bar, r->parity)) {
        next = r;
        break;
      }
    }
    if (next == nullptr) return !left;
    next->bar = nullptr;
    running = next;
    swapcontext(&scheduler, &next->at);
  }
}
}  // namespace model

// What the header takes from the instructions' header, on the model.
namespace sa {
void mbar_arrive(uint64_t* bar) { model::arrive(bar); }
bool mbar_wait_model(uint64_t* bar, uint32_t parity) {
  model::wait(bar, parity);
  return true;
}
void clc_try_cancel(uint4*, uint64_t* bar) { model::arrive(bar); }   // (no further item)
bool clc_answer(const uint4*, uint32_t&, uint32_t&, uint32_t&) { return false; }
}  // namespace sa

struct Item {
  int n, keys;
};

int main() {
  constexpr int kRing = SA_RING;
  constexpr bool kFirst = SA_FIRST;
  static uint8_t slots[kRing][kTileBytes];
  static uint64_t full[kRing], empty[kRing], cleared[kRing];
  static WorkRing work;
  static volatile uint32_t abort_flag = 0;
  static uint32_t err = 0;
  static int kv_len = 0;
  int bad = 0;
  for (int n = 1; n <= 13; ++n) {
    kv_len = n * kTile - 28;
    const Mask mask = {&kv_len, 0, kTile, 13 * kTile};
    const Item item = {n, kv_len};
    for (int s = 0; s < kRing; ++s) {
      model::init(&full[s], 1);
      model::init(&empty[s], tile_releasers(mask));
      model::init(&cleared[s], 1);
    }
    work_init(work, 1);
    for (model::Role* r : model::roles) delete r;
    model::roles.clear();
    std::vector<int> dirty(kRing, 0);   // of the tile that is in the slot: rows that have to be cleared
    int wrong = 0;
    model::add([&] {   // the load thread
      for (int j = 0; j < n; ++j) {
        const int slot = j % kRing, use = j / kRing;
        if (use > 0) model::wait(&empty[slot], (use - 1) & 1);
        std::fill(slots[slot], slots[slot] + kTileBytes, (uint8_t)1);
        model::arrive(&full[slot]);
      }
      work_request(work, 1, &abort_flag, &err);
    });
    model::add([&] {   // the MMA warp
      uint32_t parity = 0;
      for (int j = 0; j < n; ++j) {
        const int slot = j % kRing;
        model::wait(&full[slot], (j / kRing) & 1);
        if (j == (kFirst ? 0 : n - 1)) {
          model::wait(&cleared[slot], (parity >> slot) & 1);
          parity ^= 1u << slot;
          // (lane 0's pieces)
          if (slots[slot][kTileBytes / 2 - 512] != 0 || slots[slot][0] != 1) ++wrong;
        } else if (slots[slot][kTileBytes / 2 - 512] != 1) {
          ++wrong;
        }
        model::arrive(&empty[slot]);
      }
    });
    model::add([&] {
      clear_warp<kRing, kFirst>(mask, [&](const Work&) { return item; }, work, slots, full, empty, cleared, 0,
                                &abort_flag, &err);
    });
    const bool ended = model::run();
    if (!ended || wrong) {
      std::printf("ring of %d, %d tiles: %s\n", kRing, n, ended ? "a tile not cleared, or another one" : "waits for ever");
      ++bad;
    }
  }
  return bad ? 1 : 0;
}
